"""last_query_error: the first error since the last call, taken in the order of
the stream that it is given, whatever other streams are doing."""
import ctypes

import pytest
import torch

from test_gpu_query import make, pkg  # noqa: F401

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


class Calls:
    """append calls whose token `detail` has a slot outside the cache."""

    def __init__(self, pkg, s):  # noqa: F811
        self.s = s
        self.kc, self.vc = (torch.zeros(1, 4, 16, 2, 64, dtype=BF, device="cuda") for _ in range(2))
        self.cache = pkg.cache_desc(self.kc, self.vc)
        self.x = torch.zeros(4, 2, 64, dtype=BF, device="cuda")
        self.pos = torch.arange(4, device="cuda", dtype=torch.int32)
        self.slots = []
        for bad in range(4):
            t = torch.full((4,), -1, device="cuda")
            t[bad] = 64
            self.slots.append(t)
        torch.cuda.synchronize()

    def fail(self, detail, stream=None):
        self.s.append(self.x, self.x, self.pos, self.slots[detail], self.cache, stream=stream)


def test_an_error_right_after_the_last_one_is_kept(pkg):  # noqa: F811
    with make(pkg, 64, 2, layers=1) as s:
        calls = Calls(pkg, s)
        side = torch.cuda.Stream().cuda_stream
        for i in range(400):
            calls.fail(i % 4, side)
            assert s.last_query_error(side) == (pkg.IS_ERR_BAD_BLOCK, i % 4), i
        assert s.last_query_error(side) == (0, 0)


def test_it_waits_for_its_own_stream_alone(pkg):  # noqa: F811
    """Work of the default stream that is still to come neither delays the
    answer for a side stream nor loses its own error."""
    with make(pkg, 64, 2, layers=1) as s:
        calls = Calls(pkg, s)
        side = torch.cuda.Stream().cuda_stream
        torch.cuda._sleep(1_000_000_000)  # some half a second
        calls.fail(3)
        later = torch.cuda.Event()
        later.record()
        calls.fail(1, side)
        got = s.last_query_error(side)
        assert not later.query()
        assert got == (pkg.IS_ERR_BAD_BLOCK, 1)
        assert s.last_query_error(side) == (0, 0)
        assert not later.query()
        assert s.last_query_error() == (pkg.IS_ERR_BAD_BLOCK, 3)
        assert s.last_query_error() == (0, 0)


def test_the_first_of_many_is_kept_whole(pkg):  # noqa: F811
    """Code and detail belong together: details of several failing streams
    come out as one of them recorded them, each at most once a call."""
    with make(pkg, 64, 2, layers=1) as s:
        calls = Calls(pkg, s)
        streams = [torch.cuda.Stream() for _ in range(4)]
        for _ in range(100):
            for d, st in enumerate(streams):
                calls.fail(d, st.cuda_stream)
            rc, detail = s.last_query_error(streams[2].cuda_stream)
            assert rc == pkg.IS_ERR_BAD_BLOCK and detail in (0, 1, 2, 3)
            torch.cuda.synchronize()
            s.last_query_error()
        assert s.last_query_error() == (0, 0)


def test_a_refused_wait_does_not_fail_the_next_call(pkg):  # noqa: F811
    """Waiting for a stream that is being captured is an error of that call,
    and of no later one."""
    cudart = ctypes.CDLL("libcudart.so.12")
    with make(pkg, 64, 2, layers=1) as s:
        calls = Calls(pkg, s)
        st = torch.cuda.Stream()
        raw, graph = ctypes.c_void_p(st.cuda_stream), ctypes.c_void_p()
        assert cudart.cudaStreamBeginCapture(raw, 2) == 0  # relaxed
        assert s.last_query_error(st.cuda_stream)[0] == pkg.IS_ERR_CUDA
        cudart.cudaStreamEndCapture(raw, ctypes.byref(graph))
        cudart.cudaGetLastError()
        if graph.value:
            cudart.cudaGraphDestroy(graph)
        q, _ = s.rotate(calls.x, calls.pos)
        assert torch.equal(q, calls.x)
        assert s.last_query_error() == (0, 0)
