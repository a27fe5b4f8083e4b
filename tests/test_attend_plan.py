"""What an attention call launches, on the host alone: the plan of
kv_cache_injection_gather_b200/csrc/query.cu over random calls and GPUs (whole
ones, and parts of one that have room for no cluster), and stores whose GPU
gives no query handle."""
import collections
import os
import random
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
Plan = collections.namedtuple("Plan", "wide shared units splits key_parts parts shared_units ml_bytes o_bytes")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    from kv_cache_injection_gather_b200 import build
    exe = str(tmp_path_factory.mktemp("plan") / "attend_plan")
    subprocess.run(["nvcc", "-O1", "-std=c++17", *build.ARCH, "-I", os.path.join(ROOT, "include"), "-I", build.CSRC, "-o",
                    exe, os.path.join(ROOT, "tests", "c", "attend_plan.cu")], check=True)
    return exe


def plans(program, calls):
    lines = "\n".join(" ".join(str(x) for x in c) for c in calls) + "\n"
    out = subprocess.run([program], input=lines, capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(out) == len(calls)
    return [Plan(*map(int, x.split())) for x in out]


def test_a_gpu_without_room_for_large_clusters_has_fewer(program):
    out = subprocess.run([program, "clusters"], capture_output=True, text=True, check=True).stdout.splitlines()
    assert out == ["1 16 8 4 2", "1 16 8 4 0", "1 16 8 0 0", "1 16 0 0 0", "0 0 0 0 0"]


def random_call(rng):
    sms = rng.choice([148, 148, 74, 16, 2])
    largest = rng.choice([8, 8, 4, 2, 1])
    clusters = [max(1, sms // (1 << i) - rng.randrange(0, 2)) if 1 << i <= min(largest, sms) else 0 for i in range(4)]
    kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 4, 7, 8])
    requests = int(2 ** rng.uniform(0, 8))
    most = rng.choice([1, 1, 2, 5, 64, 4096])
    tokens = rng.randint(1, requests * most)
    block = rng.choice([1, 16, 24, 128])
    keys = int(2 ** rng.uniform(0, 18))
    return (sms, *clusters, kv_heads, rng.choice([32, 64, 128, 256]), tokens, requests, most, -(-keys // block),
            rng.choice([0, rng.randint(0, keys)]), kv_heads * group, block)


def test_plans_of_random_calls_hold_what_the_kernels_need(program):
    rng = random.Random(5)
    calls = [random_call(rng) for _ in range(20000)]
    seen = collections.Counter()
    for c, p in zip(calls, plans(program, calls)):
        sms, clusters, kv_heads, D, tokens = c[0], c[1:5], c[5], c[6], c[7]
        assert p.splits in (1, 2, 4, 8)
        # clusters that the GPU can run, all of them at once
        at_once = clusters[p.splits.bit_length() - 1]
        assert p.splits == 1 or (at_once > 0 and p.units * kv_heads * p.key_parts <= at_once), (c, p)
        assert 1 <= p.key_parts and 0 <= p.parts <= 32
        assert p.key_parts == 1 or p.parts == p.key_parts
        assert not p.wide or (p.splits == 1 and p.key_parts == 1 and not p.shared)
        assert not p.shared or (p.parts >= 1 and p.key_parts == 1)
        # a tile number times the shares of a unit's keys fits 32 bits
        assert p.splits * p.key_parts <= 256 and (2 ** 24) * (p.parts if p.wide or p.shared else 1) <= 2 ** 32
        rows = p.parts * tokens * c[12]
        assert p.ml_bytes == -(-rows * 8 // 256) * 256 and p.o_bytes == rows * D * 4
        seen[p.wide, p.shared, p.splits > 1, p.key_parts > 1, p.parts > 0] += 1
    assert len(seen) >= 7, seen


def test_plans_without_clusters_use_parts_alone(program):
    calls = []
    for keys in (100, 2000, 60000):
        for D in (32, 64, 128, 256):
            calls.append((16, 16, 0, 0, 0, 2, D, 3, 3, 1, keys // 16, 0, 8, 16))
    for p in plans(program, calls):
        assert p.splits == 1 and not p.wide and not p.shared


# ---------------------------------------------------------------- the store

class NoQuery:
    """The binding of a library that makes stores and no query handles."""

    def __init__(self, B):
        self.B, self.destroyed = B, []

    def __getattr__(self, name):
        return getattr(self.B, name)

    def is_store_create(self, cfg, device):
        return 4711

    def is_store_destroy(self, handle):
        self.destroyed.append(handle)

    def is_query_create(self, cfg, device):
        raise self.B.InjectError(self.B.IS_ERR_CUDA, "is_query_create")

    def is_query_destroy(self, handle):
        raise AssertionError("there is none")

    def is_store_num_facts(self, handle):
        assert handle == 4711
        return 3


def test_a_store_without_a_query_handle_still_injects(monkeypatch):
    from kv_cache_injection_gather_b200 import binding as B
    from kv_cache_injection_gather_b200 import store as S
    fake = NoQuery(B)
    monkeypatch.setattr(S, "B", fake)
    with S.FactStore(1, 2, 64, S.RopeConfig(theta=1e4), 16, 1, device=-1) as s:
        assert s.handle == 4711 and s.num_facts == 3
        x, i = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
        cache = B.is_cache_t(block_size=16)
        for call in (lambda: s.rotate(x, i, q_out=x, stream=0),
                     lambda: s.append(x, x, i, i.long(), cache, stream=0),
                     lambda: s.attend(x, torch.zeros(2, dtype=torch.int32), i, i, i[None], cache, out=x, stream=0),
                     lambda: s.last_query_error(stream=0)):
            with pytest.raises(B.InjectError) as e:
                call()
            assert e.value.status == B.IS_ERR_CUDA and "is_query_create" in str(e.value)
    assert fake.destroyed == [4711]
