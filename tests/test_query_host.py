"""The query calls' host side without a GPU: the C structs match the binding,
bad arguments are refused before any launch, the torch wrapper's checks, the
tile count bound that the launches rely on, and the fp64 references of the
GPU tests on closed forms."""
import ctypes
import math
import os
import random
import subprocess

import pytest
import torch

from query_cases import BF, Paged, attend_reference, inv_freq, rotated

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_structs_match_the_header(tmp_path):
    from kv_cache_injection_gather_b200 import binding as B
    lines = []
    for t in (B.is_rows_t, B.is_attend_t):
        lines.append(f'printf("{t.__name__} %zu\\n", sizeof({t.__name__}));')
        for name, _ in t._fields_:
            lines.append(f'printf("{t.__name__}.{name} %zu\\n", offsetof({t.__name__}, {name}));')
    src = tmp_path / "s.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "inject_query.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-o", exe, src], check=True)
    got = dict(x.split() for x in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.splitlines())
    for t in (B.is_rows_t, B.is_attend_t):
        assert int(got[t.__name__]) == ctypes.sizeof(t)
        for name, _ in t._fields_:
            assert int(got[f"{t.__name__}.{name}"]) == getattr(t, name).offset, name


def test_create_and_null_handles_are_refused():
    from kv_cache_injection_gather_b200 import binding as B
    lib = B.lib()
    out = ctypes.c_void_p()
    assert lib.is_query_create(None, 0, ctypes.byref(out)) == B.IS_ERR_INVALID_ARG
    good = dict(num_layers=1, num_kv_heads=2, head_dim=128, rope_theta=1e4)
    for change, rc in ((dict(head_dim=96), B.IS_ERR_NOT_SUPPORTED), (dict(rope_theta=0.0), B.IS_ERR_INVALID_ARG),
                       (dict(rope_theta=math.nan), B.IS_ERR_INVALID_ARG), (dict(num_layers=0), B.IS_ERR_INVALID_ARG),
                       (dict(num_kv_heads=0), B.IS_ERR_INVALID_ARG), (dict(rope_style=2), B.IS_ERR_INVALID_ARG),
                       (dict(rope_scaling=1), B.IS_ERR_INVALID_ARG), (dict(rope_scaling=5), B.IS_ERR_INVALID_ARG)):
        cfg = B.is_store_config_t(**{**good, **change})
        assert lib.is_query_create(ctypes.byref(cfg), 0, ctypes.byref(out)) == rc, change
        assert not out.value
    cfg = B.is_store_config_t(**good)
    assert lib.is_query_create(ctypes.byref(cfg), -1, ctypes.byref(out)) == B.IS_ERR_CUDA
    if not torch.cuda.is_available():
        assert lib.is_query_create(ctypes.byref(cfg), 0, ctypes.byref(out)) == B.IS_ERR_CUDA
    lib.is_query_destroy(None)  # ignored
    rows, cache, args, n = B.is_rows_t(), B.is_cache_t(), B.is_attend_t(), ctypes.c_int64()
    bad = B.IS_ERR_INVALID_ARG
    assert lib.is_query_last_error(None, None, None) == bad
    assert lib.is_query_rotate(None, 1, None, rows, rows, None, None, None, None, 0.0, None) == bad
    assert lib.is_query_append(None, 1, None, None, rows, rows, None, None, None, None, 0.0, cache, 0, None) == bad
    assert lib.is_query_attend_workspace(None, args, cache, ctypes.byref(n)) == bad
    assert lib.is_query_attend_workspace(None, args, cache, None) == bad
    assert lib.is_query_attend(None, args, cache, None, 0, None) == bad


def test_wrapper_checks_tensors():
    from kv_cache_injection_gather_b200 import store as S
    good = torch.zeros(3, 2, 64, dtype=BF)
    for t, heads, T in ((good.float(), None, 3), (good[0], None, 3), (good, 4, 3), (good, None, 4),
                        (good.transpose(0, 2), None, 3), (good, None, 3)):
        with pytest.raises(ValueError):  # the last one is not on the device
            S._rows(t, "x", heads, 64, T, 0)
    ints = torch.zeros(4, dtype=torch.int32)
    for t, n, dt in ((ints, 4, torch.int64), (ints, 5, torch.int32), (ints[::2], 2, torch.int32),
                     (ints.view(2, 2), 2, torch.int32), (ints, 4, torch.int32)):
        with pytest.raises(ValueError):
            S._ints(t, "x", n, dt, 0)


def test_tiles_fit_the_launch():
    """Units of a launch: one per request where a tile holds all its rows,
    else ceil(rows / tile) + requests; the requests' tiles never exceed it."""
    rng = random.Random(0)
    for _ in range(2000):
        R, G, tile = rng.randint(1, 60), rng.randint(1, 40), rng.choice([16, 128, 256])
        n = [rng.choice([0, 1, rng.randint(0, 300)]) for _ in range(R)]
        tiles = [-(-x * G // tile) for x in n]
        if max(n) * G <= tile:
            assert all(t <= 1 for t in tiles)
        assert sum(tiles) <= -(-sum(n) * G // tile) + R


def test_references_on_closed_forms():
    # one visible key: its value; equal keys: the mean of their values
    D, H, G = 32, 2, 3
    q = torch.randn(2, H * G, D).to(BF)
    k, v = torch.ones(2, 4, H, D).to(BF), torch.randn(2, 4, H, D).to(BF)
    out, lse, tol = attend_reference(q, [0, 2], [0], [2], torch.tensor([[1]]), k, v, 4, None, 0, True, 0.5)
    for h in range(H * G):
        assert torch.allclose(out[0, h], v[1, 0, h // G].double(), atol=1e-12)
        assert torch.allclose(out[1, h], (v[1, 0, h // G].double() + v[1, 1, h // G].double()) / 2, atol=1e-12)
        assert math.isclose(float(lse[0, h]), 0.5 * float(q[0, h].double().sum()), rel_tol=1e-12, abs_tol=1e-12)
    assert (tol >= 2.0 ** -8 * out.abs()).all()
    # rotation: position 0 is the identity, two quarter turns a negation
    x = torch.randn(2, 1, 4).to(BF)
    f = torch.tensor([math.pi, 0.0], dtype=torch.float64)
    for inter in (False, True):
        y, _ = rotated(x, None, 0.0, torch.tensor([0, 1]), f, inter)
        assert torch.allclose(y[0], x[0].double(), atol=1e-12)
        turned = [0, 1] if inter else [0, 2]
        assert torch.allclose(y[1, 0, turned], -x[1, 0, turned].double(), atol=1e-12)
    # norm: unit mean square
    y, _ = rotated(x, torch.ones(4).to(BF), 0.0, torch.tensor([0, 0]), f, False)
    assert torch.allclose((y * y).mean(-1), torch.ones(2, 1, dtype=torch.float64))
    assert torch.allclose(inv_freq(128, 5e5)[0], torch.tensor(1.0, dtype=torch.float64))


def test_paged_cases_hold_what_the_reference_reads():
    c = Paged(1, 32, 2, 2, 16, [2, 1, 0], [5, 40, 3], shared=20, device="cpu")
    out, _, _ = c.reference()
    assert torch.isfinite(out).all() and torch.isnan(c.k).any()
    assert torch.equal(torch.nan_to_num(c.k_cache[1]), torch.nan_to_num(c.k)) and torch.isnan(c.k_cache[0]).all()
