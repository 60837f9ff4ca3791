"""What the library's calls share with the rest of the process: the CUDA runtime's error state."""
import ctypes

import numpy as np
import pytest

import csr_spmm_gb300 as cs
from synth import power_law
from synth.fw import fw_random
from synth.workloads import tiny_uniform

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _runtime():
    """The CUDA runtime that this process has loaded."""
    cs.library()
    torch.zeros(1, device="cuda")
    with open("/proc/self/maps") as f:
        paths = {line.split()[-1] for line in f if "libcudart" in line}
    assert len(paths) == 1, f"one runtime for torch and the library: {paths}"
    return ctypes.CDLL(paths.pop())


def _products():
    """Calls of the sparse operators that reach their kernels, by name: each returns its status."""
    small, large = tiny_uniform(), power_law(30_000, 30_000, 64, 600_000, 10_000, seed=5)
    calls = {}
    for name, p in (("small", small), ("rows", large)):
        rp, ci, va, B, C = (_t(a) for a in (p.row_ptr, p.col_idx, p.values, p.B, p.C0))
        keep = (rp, ci, va, B, C)
        args = (p.alpha, rp.data_ptr(), ci.data_ptr(), va.data_ptr(), p.m, p.k, B.data_ptr(),
                p.ldb, p.n, p.beta, C.data_ptr(), p.ldc)
        calls[name] = lambda h, a=args, k=keep: cs.spmm_csr_f32(h.ptr, *a, check=False)
        scale = (0.0,) + args[1:]
        calls[name + " alpha 0"] = lambda h, a=scale, k=keep: cs.spmm_csr_f32(h.ptr, *a,
                                                                              check=False)
    for k in (20, 120):                                 # on the tensor cores, and not
        f = fw_random(300, k, 6, seed=3)
        mats = [tuple(_t(x) for x in m) for m in (f.k2b, f.t1, f.t2, f.b)]
        outs = (torch.empty(k, device="cuda"), torch.empty(k, dtype=torch.int32, device="cuda"),
                torch.empty(1, device="cuda"))
        keep = (mats, outs)
        args = (300, k, *(tuple(x.data_ptr() for x in m) for m in mats),
                *(o.data_ptr() for o in outs))
        calls[f"fw_argmin {k}"] = lambda h, a=args, k=keep: cs.spmm_fw_argmin(h.ptr, *a, check=False)
    n = 4
    rp = _t(np.arange(n + 1, dtype=np.int32))
    ci, va = _t(np.arange(n, dtype=np.int32)), _t(np.full(n, 2.0, np.float32))
    status = _t(np.zeros(1, np.int32))
    calls["ilu0"] = lambda h: cs.spmm_ilu0(h.ptr, n, n, rp.data_ptr(), ci.data_ptr(),
                                           va.data_ptr(), 0, status.data_ptr(), check=False)
    return calls


def _operators():
    """Calls of the language-model operators through C, by name: each returns its status."""
    x = torch.randn(40, 104, device="cuda")
    y, f = torch.empty_like(x), torch.ones(104, device="cuda")
    ids = torch.arange(40, device="cuda", dtype=torch.int32) % 7
    keep = (x, y, f, ids)
    a, o, v, i = x.data_ptr(), y.data_ptr(), f.data_ptr(), ids.data_ptr()
    off = o + 4
    return {
        "embedding": lambda h, k=keep: cs.spmm_embedding(h.ptr, 0, 1.0, i, 40, a, 104, 40, 104, o,
                                                         104, check=False),
        "embedding shifted": lambda h: cs.spmm_embedding(h.ptr, 0, 1.0, i, 39, a, 104, 40, 101,
                                                         off, 104, check=False),
        "embedding_grad": lambda h: cs.spmm_embedding_grad(h.ptr, 0, 0, 1.0, i, 40, a, 104, 0.0, o,
                                                           104, 40, 104, check=False),
        "layer_norm": lambda h: cs.spmm_layer_norm(h.ptr, 0, 0, a, 104, 40, 104, v, v, 1e-5, o,
                                                   104, 0, 0, check=False),
        "layer_norm apart": lambda h: cs.spmm_layer_norm(h.ptr, 0, 0, a, 104, 39, 100, v, v, 1e-5,
                                                         off, 104, 0, 0, check=False),
        "layer_norm_grad": lambda h: cs.spmm_layer_norm_grad(
            h.ptr, 0, 0, a, 104, a, 104, v, v, v, 40, 104, o, 104, 0, 0, check=False),
        "layer_norm_grad apart": lambda h: cs.spmm_layer_norm_grad(
            h.ptr, 0, 0, a, 104, a, 104, v, v, v, 39, 100, off, 104, 0, 0, check=False),
        "token_logprob": lambda h: cs.spmm_token_logprob(h.ptr, 0, 1.0, a, 104, 40, 104, i, 0, o,
                                                         0, 0, 0, 0, check=False),
        "token_logprob_grad": lambda h: cs.spmm_token_logprob_grad(
            h.ptr, 0, 1.0, a, 104, 40, 104, i, v, 0, v, 0, o, 104, check=False),
    }


def test_an_error_left_pending_is_the_callers():
    """A runtime error that the caller has not looked at is neither reported as a call's nor
    taken away by it: the library shares the process's runtime and its error state."""
    rt = _runtime()
    with cs.Handle(0) as h:
        calls = {**_products(), **_operators()}
        torch.cuda.synchronize()
        failed, gone = [], []
        for name, call in calls.items():
            assert call(h) == cs.SPMM_OK, name          # scratch in place
            torch.cuda.synchronize()
            pending = rt.cudaSetDevice(1 << 20)         # refused on the host: no such device
            assert pending != 0 and rt.cudaPeekAtLastError() == pending
            if call(h) != cs.SPMM_OK:
                failed.append(name)
            if rt.cudaGetLastError() != pending:
                gone.append(name)
            torch.cuda.synchronize()
        assert (failed, gone) == ([], [])
        other = cs.Handle(0)
        rt.cudaSetDevice(1 << 20)
        other.close()
        assert rt.cudaGetLastError() == pending, "destroying a handle"
