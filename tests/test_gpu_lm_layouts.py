"""Row layouts whose number of warps is no power of two, and scratch reserved for every
smaller call."""
import numpy as np
import pytest

import lm_reference as ref
from test_gpu_lm import _make, _near, _np, _vec, cs, handle  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [5, 700, 3000])
@pytest.mark.parametrize("dim", [768, 1536, 2560, 3008, 5120, 6144])
@pytest.mark.parametrize("t,pt", [("f32", "f32"), ("f16", "f16"), ("bf16", "f32")])
def test_norms_of_aligned_rows(cs, handle, t, pt, dim, rows):  # noqa: F811
    """Aligned rows take as many warps as they need: 3, 5, 6, 10 or 12 of them, several rows
    to a block or one."""
    rng = np.random.default_rng(rows + dim)
    x, h_x = _make(rng, (rows, dim), t, 1.5, 0.7)
    w, h_w = _vec(rng, dim, pt, 0.3, 1.0)
    b, h_b = _vec(rng, dim, pt, 0.2)
    eps = float(np.float32(1e-3))
    got = cs.layer_norm(handle, x, w, b, eps=1e-3)
    for g, (want, bound), what in zip(got, ref.layer_norm(h_x, h_w, h_b, eps, t),
                                      ("y", "mean", "rstd")):
        _near(_np(g), want, bound, what)
    dy, h_dy = _make(rng, (rows, dim), t, 0.5, 0.1)
    mean, rstd = got[1], got[2]
    grads = cs.layer_norm_grad(handle, dy, x, mean, rstd, w)
    for g, (want, bound), what in zip(
            grads, ref.layer_norm_grad(h_dy, h_x, _np(mean), _np(rstd), h_w, t, pt),
            ("dx", "dweight", "dbias")):
        _near(_np(g), want, bound, what)


@pytest.mark.parametrize("rows,dim", [(1, 1), (300, 40), (4096, 256), (4097, 264), (8193, 100),
                                      (20000, 1000), (700, 8200), (9, 20001)])
def test_a_reserve_covers_every_smaller_call(cs, rows, dim):  # noqa: F811
    """No call of up to that size allocates: within a capture it could not."""
    sizes = sorted({min(rows, n) for n in (1, 2, 31, 255, 2048, 4095, 4096, 4097, 8192, 8193,
                                           20000, rows)})
    widths = sorted({min(dim, d) for d in (1, 7, 8, 9, 255, 256, 257, 264, 513, 1000, 8192, dim)})
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    a = torch.zeros(rows, dim, device="cuda")
    stats = torch.zeros(rows, device="cuda")
    dx, table = torch.empty_like(a), torch.empty(3, dim, device="cuda")
    dw = torch.empty(dim, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with cs.Handle(0) as h:
        h.reserve_lm(rows, dim)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            st = torch.cuda.current_stream().cuda_stream
            for n in sizes:
                for d in widths:
                    cs.spmm_embedding_grad(h.ptr, 0, 0, 1.0, ids.data_ptr(), n, a.data_ptr(), dim,
                                           0.0, table.data_ptr(), dim, 3, d, st)
                    cs.spmm_layer_norm_grad(h.ptr, 0, 0, a.data_ptr(), dim, a.data_ptr(), dim,
                                            stats.data_ptr(), stats.data_ptr(), dw.data_ptr(), n,
                                            d, dx.data_ptr(), dim, dw.data_ptr(), 0, st)
        torch.cuda.synchronize()
