"""Host threads with handles of their own, in calls of different sizes."""
import threading

import numpy as np
import pytest

import csr_spmm_gb300 as cs
from synth.fw import fw_random

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def test_host_threads_with_calls_of_different_sizes():
    """A kernel's shared-memory limit belongs to the process: a call of one host thread must
    not lower it between another's setting and launch."""
    errors = []
    start = threading.Barrier(4)

    def run(make):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream), cs.Handle(0) as h:
                call = make(h)
                call()
                stream.synchronize()
                start.wait()
                for i in range(3000):
                    call()
                    if i % 100 == 99:
                        stream.synchronize()
        except Exception as e:                          # noqa: BLE001
            errors.append(e)
            start.abort()

    def norms(dim, odd):
        def make(h):
            x = torch.randn(8, dim, device="cuda")
            dx, stats = torch.empty_like(x), torch.ones(8, device="cuda")
            edges = torch.randn(400, odd, device="cuda")
            y, w = torch.empty_like(edges), torch.ones(max(dim, odd), device="cuda")
            a, b, c, s = x.data_ptr(), w.data_ptr(), edges.data_ptr(), stats.data_ptr()

            def call():
                st = torch.cuda.current_stream().cuda_stream
                cs.spmm_layer_norm_grad(h.ptr, 0, 0, a, dim, a, dim, s, s, b, 8, dim,
                                        dx.data_ptr(), dim, 0, 0, st)
                cs.spmm_layer_norm(h.ptr, 0, 0, c, odd, 400, odd, b, b, 1e-5, y.data_ptr(), odd,
                                   0, 0, st)
            return call
        return make

    def scans(k):
        def make(h):
            f = fw_random(300, k, 6, seed=3)
            mats = [tuple(_t(x) for x in m) for m in (f.k2b, f.t1, f.t2, f.b)]
            return lambda: cs.fw_argmin(h, f.k, *mats)
        return make

    threads = [threading.Thread(target=run, args=(m,))
               for m in (norms(1024, 5001), norms(4096, 9001), scans(20), scans(100))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert errors == []
