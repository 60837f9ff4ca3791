"""Captured graphs and the scratch of the handle that their calls were made on."""
import numpy as np
import pytest

import csr_spmm_gb300 as cs
from synth import power_law

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build_library()


def _t(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def test_a_captured_graph_keeps_its_scratch():
    """A later, larger call grows the handle's scratch; what a graph captured before holds
    stays its own until the handle goes."""
    torch.manual_seed(2)
    vocab, dim, n = 400, 520, 700
    ids = torch.randint(0, vocab, (n,), device="cuda", dtype=torch.int32)
    d = torch.randn(n, dim, device="cuda")
    stats = torch.rand(n, device="cuda") + 0.5
    w = torch.rand(dim, device="cuda")
    p = power_law(30_000, 30_000, 64, 600_000, 10_000, seed=5)
    rp, ci, va, B = (_t(a) for a in (p.row_ptr, p.col_idx, p.values, p.B))
    C0 = _t(p.C0)
    with cs.Handle(0) as h:
        h.reserve_lm(n, dim)
        h.reserve(p.m, p.n, 4)
        table, C = torch.empty(vocab, dim, device="cuda"), C0.clone()
        out = []

        def calls():
            cs.embedding_grad(h, ids, d, table, scale=2.0)
            out[:] = cs.layer_norm_grad(h, d, d, stats, stats, w)
            cs.spmm(h, p.alpha, rp, ci, va, p.k, B, p.beta, C)

        calls()
        torch.cuda.synchronize()
        want = [t.clone() for t in (table, *out, C)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
        held = [table, *out, C]
        # larger calls: both scratch buffers grow, twice
        for more in (8, 20):
            big = torch.randn(more * n, 4 * dim, device="cuda")
            many = ids.repeat(more)
            cs.embedding_grad(h, many, big, torch.empty(vocab, 4 * dim, device="cuda"))
            cs.layer_norm_grad(h, big, big, stats.repeat(more), stats.repeat(more))
            wide = torch.randn(p.k, 2 * more * p.n, device="cuda")
            cs.spmm(h, 1.0, rp, ci, va, p.k, wide, 0.0,
                    torch.empty(p.m, wide.shape[1], device="cuda"))
            torch.cuda.synchronize()
        # memory of the old buffers' sizes for others, were they given back
        others = [torch.full((s << 18,), float("nan"), device="cuda") for s in (1, 2, 4, 8, 16, 32)]
        for _ in range(2):
            for t in held:
                t.zero_()
            C.copy_(C0)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, held))
        assert all(bool(o.isnan().all()) for o in others)


def test_growth_gives_back_what_no_graph_holds():
    """Only buffers that a captured call has used outlive their growth."""
    rows = 4096

    def grad(h, dim):
        x = torch.randn(rows, dim, device="cuda")
        stats = torch.ones(rows, device="cuda")
        cs.layer_norm_grad(h, x, x, stats, stats)

    with cs.Handle(0) as h:
        for dim in (1024, 2048, 4096, 8192):            # about 20 KB of scratch per column
            grad(h, dim)
            torch.cuda.synchronize()
        torch.cuda.empty_cache()
        held = torch.cuda.mem_get_info()[0]
        h.close()
        torch.cuda.synchronize()
        freed = torch.cuda.mem_get_info()[0] - held
    # parts of 8192 columns for at most 16 slices per SM, a quarter more, in 2 MB pages; what
    # the smaller calls had would add 7/8 of it
    most = 1.25 * (8 * 8192 * 16 * torch.cuda.get_device_properties(0).multi_processor_count
                   + 8 * rows)
    assert 0 < freed <= most + (8 << 20)
