"""The language-model operators on the GPU against their definitions in 64 bits.

Bounds come from lm_reference (binary32 sums, one final rounding)."""
import numpy as np
import pytest

import lm_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TYPES = ("f32", "f16", "bf16")


@pytest.fixture(scope="module")
def cs():
    import __graft_entry__
    __graft_entry__.build_library()
    import csr_spmm_gb300
    return csr_spmm_gb300


@pytest.fixture(scope="module")
def handle(cs):
    h = cs.Handle(0)
    yield h
    h.close()


def _make(rng, shape, t, scale=1.0, shift=0.0, pad=0, offset=0):
    """(CUDA tensor of `shape` with row stride shape[1] + pad, starting `offset`
    elements into its buffer; its values in 64 bits)."""
    rows, cols = shape
    buf = torch.full((offset + rows * (cols + pad) + pad,), float("nan"), dtype=DT[t])
    view = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(torch.from_numpy(rng.standard_normal(shape) * scale + shift))
    dev = buf.cuda()
    out = dev[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    return out, view.double().numpy()


def _like(x, offset):
    """An uninitialised matrix that lies in its buffer as `x`, made with `offset`, does."""
    rows, ld = x.shape[0], x.stride(0)
    buf = torch.empty(offset + rows * ld, dtype=x.dtype, device="cuda")
    return buf[offset:].view(rows, ld)[:, :x.shape[1]]


def _vec(rng, n, t, scale=1.0, shift=0.0):
    v, h = _make(rng, (1, n), t, scale, shift)
    return v[0].contiguous(), h[0]


def _np(t):
    return t.double().cpu().numpy()


def _near(got, want, bound, what=""):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    same = (np.isnan(got) & np.isnan(want)) | (got == want)
    with np.errstate(invalid="ignore"):
        ok = same | (np.abs(got - want) <= bound)
    if not ok.all():
        at = tuple(np.argwhere(~ok)[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.size} off, first at {at}: got "
                             f"{got[at]!r}, want {want[at]!r}, bound {np.broadcast_to(bound, want.shape)[at]!r}")


# ---- embedding -----------------------------------------------------------------

@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("tokens,vocab,dim,pad,offset", [
    (1, 1, 1, 0, 0), (1, 50, 8, 0, 0), (2, 7, 7, 0, 0), (37, 100, 64, 8, 0), (1000, 300, 100, 0, 0),
    (513, 999, 1001, 0, 0), (64, 40, 2048, 0, 1), (9, 33, 8200, 0, 0), (3, 5, 70001, 3, 0),
    (20000, 1000, 24, 0, 0), (700, 300, 4096, 0, 0)])
def test_embedding(cs, handle, t, tokens, vocab, dim, pad, offset):
    """One binary32 product, rounded once: equal bit for bit."""
    rng = np.random.default_rng(tokens * 31 + dim)
    table, _ = _make(rng, (vocab, dim), t, pad=pad, offset=offset)
    ids = rng.integers(-2, vocab + 2, tokens).astype(np.int32)
    ids[0] = vocab - 1
    scale = float(np.float32(3.7))
    d_ids = torch.from_numpy(ids).cuda()
    got = cs.embedding(handle, d_ids, table, scale=scale)
    ok = torch.from_numpy((ids >= 0) & (ids < vocab)).cuda()
    want = (table[torch.where(ok, d_ids, 0).long()].float() * scale) * ok[:, None]
    assert torch.equal(got, want.to(DT[t]))
    out = torch.full((tokens, dim + 5), 7.0, dtype=DT[t], device="cuda")
    assert cs.embedding(handle, d_ids, table, scale=scale, out=out[:, :dim]) is not None
    assert torch.equal(out[:, :dim], got) and bool((out[:, dim:] == 7.0).all())


def test_embedding_edges(cs, handle):
    table = torch.randn(5, 16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert cs.embedding(handle, none, table).shape == (0, 16)
    assert cs.embedding(handle, none, table[:, :0]).shape == (0, 0)
    ids = torch.tensor([0, 4, -1, 5, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    got = cs.embedding(handle, ids, table)
    assert torch.equal(got[:2], table[[0, 4]]) and not bool(got[2:].any())
    assert not bool(cs.embedding(handle, ids, table[:0]).any())        # no vocabulary
    table[4, 3] = float("nan")
    assert not bool(cs.embedding(handle, ids, table, scale=0.0).any())  # not read
    assert bool(cs.embedding(handle, ids, table)[1].isnan()[3])


# ---- the embedding's gradient -----------------------------------------------------

def _zipf_ids(rng, tokens, vocab):
    p = 1.0 / (np.arange(vocab) + 2.7)
    ids = rng.permutation(vocab)[rng.choice(vocab, tokens, p=p / p.sum())]
    return ids.astype(np.int32)


@pytest.mark.parametrize("t,gt", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"),
                                  ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("tokens,vocab,dim,beta,pad,offset", [
    (1, 1, 1, 0.0, 0, 0), (1, 300, 8, 0.0, 0, 0), (2, 5, 33, 1.0, 0, 0), (33, 1000, 64, 0.5, 0, 0),
    (65, 3, 256, 1.0, 8, 0), (384, 5000, 1001, 1.0, 0, 0), (4095, 200, 40, 0.0, 0, 1),
    (4096, 4096, 16, -1.0, 0, 0), (4097, 1, 24, 0.0, 0, 0), (9000, 700, 136, 1.0, 0, 0),
    (70001, 2000, 8, 0.0, 0, 0), (70001, 40000, 3, 1.0, 0, 0), (300, 100, 5000, 0.0, 0, 0)])
def test_embedding_grad(cs, handle, t, gt, tokens, vocab, dim, beta, pad, offset):
    rng = np.random.default_rng(tokens + dim)
    ids = _zipf_ids(rng, tokens, vocab)
    if tokens > 8:
        ids[rng.random(tokens) < 0.1] = rng.choice([-1, vocab, -2 ** 31, 2 ** 31 - 1])
    dout, h_dout = _make(rng, (tokens, dim), t, 0.3, pad=pad, offset=offset)
    dtable, h_old = _make(rng, (vocab, dim), gt, 0.5, pad=pad, offset=offset)
    if beta == 0.0:
        dtable.fill_(float("nan"))                     # must not be read
    again = dtable.clone()
    scale = float(np.float32(1.75))
    d_ids = torch.from_numpy(ids).cuda()
    cs.embedding_grad(handle, d_ids, dout, dtable, scale=scale, beta=beta)
    want, bound = ref.embedding_grad(ids, h_dout, h_old, scale, beta, gt)
    _near(_np(dtable), want, bound, "dtable")
    cs.embedding_grad(handle, d_ids, dout.contiguous(), again, scale=scale, beta=beta)
    assert torch.equal(again, dtable), "another layout of the same values gives other bits"


@pytest.mark.parametrize("tokens,lengths", [
    (1000, [1000]), (6000, [5000, 1000]), (300, [31, 1, 32, 33, 64, 1, 1, 128, 9]),
    (70000, [1, 69998, 1]), (200000, [65536, 100000, 34464])])
def test_embedding_grad_long_runs(cs, handle, tokens, lengths):
    """Runs of one id that span pieces of every kind, in a shuffled order."""
    rng = np.random.default_rng(tokens)
    vocab = 2 * len(lengths) + 1
    ids = np.repeat(2 * np.arange(len(lengths)) + 1, lengths).astype(np.int32)
    assert ids.size == tokens
    rng.shuffle(ids)
    for dim, t in ((8, "f32"), (300, "bf16")):
        dout, h_dout = _make(rng, (tokens, dim), t, 0.3)
        dtable = torch.full((vocab, dim), float("nan"), device="cuda")
        cs.embedding_grad(handle, torch.from_numpy(ids).cuda(), dout, dtable)
        want, bound = ref.embedding_grad(ids, h_dout, np.zeros((vocab, dim)), 1.0, 0.0, "f32")
        _near(_np(dtable), want, bound, "dtable")


def test_embedding_grad_edges(cs, handle):
    dt = torch.randn(6, 16, device="cuda")
    old = dt.clone()
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    cs.embedding_grad(handle, none, torch.empty(0, 16, device="cuda"), dt, beta=1.0)
    assert torch.equal(dt, old)
    cs.embedding_grad(handle, none, torch.empty(0, 16, device="cuda"), dt, beta=0.5)
    assert torch.equal(dt, 0.5 * old)
    ids = torch.tensor([-1, 6, -5], dtype=torch.int32, device="cuda")
    d = torch.full((3, 16), float("nan"), device="cuda")
    cs.embedding_grad(handle, ids, d, dt, beta=1.0)            # only padding: not summed
    assert torch.equal(dt, 0.5 * old)
    ids[0] = 2
    cs.embedding_grad(handle, ids, d, dt, scale=0.0, beta=1.0)  # dout not read
    assert torch.equal(dt, 0.5 * old)
    cs.embedding_grad(handle, ids, d, dt, beta=0.0)
    assert bool(dt[2].isnan().all()) and not bool(dt[[0, 1, 3, 4, 5]].any())
    cs.embedding_grad(handle, ids, d, dt, scale=0.0, beta=0.0)
    assert not bool(dt.any())
    cs.embedding_grad(handle, ids, d[:, :0], dt[:, :0])
    cs.embedding_grad(handle, ids, d, dt[:0])


def test_embedding_gradient_against_differences(cs, handle):
    """d/dtable of sum(out * c), out the lookup: central differences in 64 bits."""
    rng = np.random.default_rng(5)
    ids = np.array([3, 0, 3, -1, 2, 3, 9], np.int32)
    c, h_c = _make(rng, (7, 4), "f32")
    table = rng.standard_normal((5, 4))
    ok = (ids >= 0) & (ids < 5)

    def loss(tab):
        return float((2.5 * tab[np.where(ok, ids, 0)] * ok[:, None] * h_c).sum())

    got = torch.empty(5, 4, device="cuda")
    cs.embedding_grad(handle, torch.from_numpy(ids).cuda(), c, got, scale=2.5)
    _against_differences(loss, table, _np(got))


def _against_differences(loss, at, grad, step=1e-5):
    """Central differences in 64 bits: off by step^2 of the third derivative and
    the losses' rounding over the step, both far below 1e-5 here."""
    want = np.zeros_like(at)
    for i in np.ndindex(at.shape):
        up, down = at.copy(), at.copy()
        up[i] += step
        down[i] -= step
        want[i] = (loss(up) - loss(down)) / (2 * step)
    _near(grad, want, 1e-5 * (1 + np.abs(want)), "differences")


# ---- layer norm ----------------------------------------------------------------

SHAPES = [(1, 1, 0, 0), (3, 2, 0, 0), (5, 31, 0, 0), (130, 64, 0, 0), (4, 256, 8, 0),
          (1000, 128, 0, 0), (33, 1000, 0, 1), (70, 1001, 0, 0), (9, 2048, 0, 0),
          (513, 520, 16, 0), (40, 4096, 0, 0), (7, 5000, 3, 0), (12, 8192, 0, 0),
          (3, 8200, 0, 0), (5, 16384, 0, 0), (2, 20000, 0, 0), (2, 70001, 0, 0),
          (1, 40960, 0, 0), (3000, 48, 0, 0), (4000, 7, 0, 0), (9000, 3, 0, 1), (2600, 515, 0, 0),
          (1300, 2048, 0, 0), (700, 8200, 1, 0), (350, 16391, 0, 0), (2, 65536, 0, 0)]


@pytest.mark.parametrize("t,pt", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"),
                                  ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,dim,pad,offset", SHAPES)
def test_layer_norm(cs, handle, t, pt, rows, dim, pad, offset):
    rng = np.random.default_rng(rows + dim)
    x, h_x = _make(rng, (rows, dim), t, 1.5, 0.7, pad=pad, offset=offset)
    w, h_w = _vec(rng, dim, pt, 0.3, 1.0)
    b, h_b = _vec(rng, dim, pt, 0.2)
    got = cs.layer_norm(handle, x, w, b, eps=1e-3)
    for g, (want, bound), what in zip(got, ref.layer_norm(h_x, h_w, h_b, float(np.float32(1e-3)),
                                                          t), ("y", "mean", "rstd")):
        _near(_np(g), want, bound, what)
    plain = cs.layer_norm(handle, x, eps=1e-3)
    _near(_np(plain[0]), *ref.layer_norm(h_x, 1.0, 0.0, float(np.float32(1e-3)), t)[0], "no weight")
    apart = cs.layer_norm(handle, x, w, b, eps=1e-3, out=_like(x, offset))[0]
    y = cs.layer_norm(handle, x, w, b, eps=1e-3, out=x)[0]
    assert y.data_ptr() == x.data_ptr() and torch.equal(y, apart), "in place"
    _near(_np(y), *ref.layer_norm(h_x, h_w, h_b, float(np.float32(1e-3)), t)[0], "in place")


@pytest.mark.parametrize("dim", [64, 1001, 4096, 20000])
def test_layer_norm_far_from_zero(cs, handle, dim):
    """A mean 1000 times the deviation: a one-pass variance would lose it."""
    rng = np.random.default_rng(dim)
    x, h_x = _make(rng, (5, dim), "f32", 0.01, 10.0)
    got = cs.layer_norm(handle, x, eps=0.0)
    for g, (want, bound), what in zip(got, ref.layer_norm(h_x, 1.0, 0.0, 0.0, "f32"),
                                      ("y", "mean", "rstd")):
        _near(_np(g), want, bound, what)


def test_layer_norm_edges(cs, handle):
    x = torch.full((3, 40), 2.5, device="cuda")
    y, mean, rstd = cs.layer_norm(handle, x, eps=0.25)
    assert not bool(y.any()) and bool((mean == 2.5).all()) and bool((rstd == 2.0).all())
    y, _, rstd = cs.layer_norm(handle, x, eps=0.0)              # 0 * inf, as the formula
    assert bool(y.isnan().all()) and bool(rstd.isinf().all())
    x[1, 7] = float("nan")
    y, _, _ = cs.layer_norm(handle, x, eps=0.25)
    assert bool(y[1].isnan().all()) and not bool(y[[0, 2]].any())
    y, mean, rstd = cs.layer_norm(handle, x[:0])
    assert y.shape == (0, 40) and mean.shape == rstd.shape == (0,)
    assert cs.layer_norm(handle, x[:, :0])[0].shape == (3, 0)
    dx, dw, db = cs.layer_norm_grad(handle, x[:0], x[:0], mean, rstd,
                                    torch.ones(40, device="cuda"))
    assert dx.shape == (0, 40) and not bool(dw.any()) and not bool(db.any())


@pytest.mark.parametrize("t,pt", [("f32", "f32"), ("f16", "f16"), ("f16", "f32"),
                                  ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,dim,pad,offset", SHAPES)
def test_layer_norm_grad(cs, handle, t, pt, rows, dim, pad, offset):
    rng = np.random.default_rng(rows + 7 * dim)
    x, h_x = _make(rng, (rows, dim), t, 1.5, 0.7, pad=pad, offset=offset)
    dy, h_dy = _make(rng, (rows, dim), t, 0.5, 0.1, pad=pad)
    w, h_w = _vec(rng, dim, pt, 0.3, 1.0)
    mean, h_mean = _vec(rng, rows, "f32", 0.1, 0.7)
    rstd, h_rstd = _vec(rng, rows, "f32", 0.05, 0.6)
    got = cs.layer_norm_grad(handle, dy, x, mean, rstd, w)
    want = ref.layer_norm_grad(h_dy, h_x, h_mean, h_rstd, h_w, t, pt)
    for g, (v, bound), what in zip(got, want, ("dx", "dweight", "dbias")):
        _near(_np(g), v, bound, what)
    plain = cs.layer_norm_grad(handle, dy, x, mean, rstd, bias=False)
    assert plain[1] is None and plain[2] is None
    _near(_np(plain[0]), *ref.layer_norm_grad(h_dy, h_x, h_mean, h_rstd, 1.0, t, pt)[0], "dx")
    apart = cs.layer_norm_grad(handle, dy, x, mean, rstd, w, out=_like(dy, 0))
    again = cs.layer_norm_grad(handle, dy, x, mean, rstd, w, out=dy)
    for a, b in zip(again, apart):
        assert torch.equal(a, b), "in place, and the same bits again"
    for g, (v, bound), what in zip(again, want, ("dx", "dweight", "dbias")):
        _near(_np(g), v, bound, what)


def test_layer_norm_gradient_against_differences(cs, handle):
    rng = np.random.default_rng(8)
    x, h_x = _make(rng, (4, 9), "f32", 1.5, 0.5)
    w, h_w = _vec(rng, 9, "f32", 0.3, 1.0)
    b, h_b = _vec(rng, 9, "f32")
    dy, h_dy = _make(rng, (4, 9), "f32")
    _, mean, rstd = cs.layer_norm(handle, x, w, b, eps=1e-5)
    dx, dw, db = cs.layer_norm_grad(handle, dy, x, mean, rstd, w)

    def loss(xx, ww, bb):
        return float((ref.layer_norm(xx, ww, bb, float(np.float32(1e-5)), "f32")[0][0]
                      * h_dy).sum())

    _against_differences(lambda v: loss(v, h_w, h_b), h_x, _np(dx))
    _against_differences(lambda v: loss(h_x, v, h_b), h_w, _np(dw))
    _against_differences(lambda v: loss(h_x, h_w, v), h_b, _np(db))


# ---- token log probabilities ------------------------------------------------------

def _check_logprob(cs, handle, x, h_x, targets, alpha, k):
    d_t = None if targets is None else torch.from_numpy(targets).cuda()
    got = cs.token_logprob(handle, x, d_t, alpha=alpha, top=k)
    a32 = float(np.float32(alpha))
    want, tol = ref.token_logprob(h_x, targets, a32)
    assert (got[0] is None) == (targets is None)
    for g, name in zip(got[:3], ("logprob", "entropy", "lse")):
        if g is not None:
            _near(_np(g), want[name], tol[name], name)
    if k:
        index = ref.top(h_x, k)
        assert np.array_equal(got[4].cpu().numpy(), index), "top_index"
        picked = np.take_along_axis(h_x, np.maximum(index, 0), 1) if h_x.shape[1] else \
            np.zeros(index.shape)
        with np.errstate(invalid="ignore"):
            lp = np.where(index >= 0, a32 * picked - want["lse"][:, None], -np.inf)
        lp[np.isnan(want["lse"])] = np.nan
        with np.errstate(invalid="ignore"):
            bound = tol["lse"][:, None] + ref.U * (2 * np.abs(a32 * picked) + np.abs(lp))
        _near(_np(got[3]), lp, bound, "top_logprob")
    return got


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,vocab,k,alpha,pad,offset", [
    (1, 1, 1, 1.0, 0, 0), (3, 2, 5, 0.5, 0, 0), (4, 31, 32, 1.0, 0, 0), (5, 100, 8, 1.0, 0, 0),
    (2, 1000, 20, 1.25, 8, 0), (33, 1001, 5, 1.0, 0, 0), (7, 4096, 32, 1.0, 0, 3),
    (9, 5003, 0, 2.0, 5, 0), (200, 2048, 1, 1.0, 0, 0), (170, 10007, 10, 0.7, 0, 1),
    (3, 50001, 20, 1.0, 0, 0), (1, 131072, 8, 1.0, 0, 0), (2, 300000, 32, 1.0, 0, 0),
    (400, 777, 3, 1.0, 0, 0)])
def test_token_logprob(cs, handle, t, rows, vocab, k, alpha, pad, offset):
    rng = np.random.default_rng(rows * 7 + vocab)
    x, h_x = _make(rng, (rows, vocab), t, 3.0, pad=pad, offset=offset)
    targets = rng.integers(-1, vocab + 1, rows).astype(np.int32)
    targets[0] = vocab - 1
    got = _check_logprob(cs, handle, x, h_x, targets, alpha, k)
    again = cs.token_logprob(handle, x, torch.from_numpy(targets).cuda(), alpha=alpha, top=k)
    assert all(torch.equal(a, b) for a, b in zip(got, again)), "the same bits again"


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("vocab,times", [(5, 1), (64, 1), (300, 1), (1001, 1), (9000, 1),
                                         (70000, 1), (1001, 60), (9003, 60), (40001, 60)])
def test_token_logprob_masks_and_special_values(cs, handle, t, vocab, times):
    """Rows with masked, lowest, equal, infinite and NaN logits: few rows, and the same
    rows `times` over (every copy must give the same bits)."""
    rng = np.random.default_rng(vocab)
    x, _ = _make(rng, (14, vocab), t, 2.0)
    low = float(torch.finfo(DT[t]).min)
    inf = float("inf")
    last = vocab - 1
    x[0] = -inf                                        # nothing left
    x[1] = -inf
    x[1, last] = 1.5                                   # one left
    x[2] = low                                         # the type's lowest value everywhere
    x[3] = low
    x[3, vocab // 2] = 2.0
    x[4] = 0.25                                        # all equal: ties by lowest index
    x[5, ::2] = -0.0
    x[5, 1::2] = 0.0                                   # -0 and 0 tie
    x[6, vocab // 3] = float("nan")
    x[7, last] = inf
    x[8, : vocab - 3] = -inf                           # three left, at the end
    x[9, 0] = -float("nan") if vocab < 300 else float("nan")
    x[9, last] = -inf
    x[10] = -float(torch.finfo(DT[t]).max)
    x[10, 0] = -inf
    x[11] = float(torch.finfo(DT[t]).max)              # the largest value everywhere
    x[12] = torch.randint(0, 2, (vocab,), device="cuda").to(DT[t])   # two values: many ties
    x[13, ::3] = -inf
    if times > 1:
        many = x.repeat(times, 1)
        targets = torch.full((14 * times,), last, dtype=torch.int32, device="cuda")
        for k in (0, 4, 32):
            got = cs.token_logprob(handle, many, targets, top=k)
            ld = many.stride(0) * many.element_size()
            for g in got:
                g = g.view(times, 14, -1)
                # copies that lie alike against 16-byte boundaries
                step = 16 // np.gcd(16, 14 * ld)
                want = g[:step].repeat(-(-times // step), 1, 1)[:times]
                same = (g == want) | ((g != g) & (want != want))
                assert bool(same.all())
            first = [g[:14].double().cpu().numpy() for g in got]
            want, tol = ref.token_logprob(_np(x), targets[:14].cpu().numpy(), 1.0)
            for g, name in zip(first, ("logprob", "entropy", "lse")):
                _near(g, want[name], tol[name], name)
            if k:
                assert np.array_equal(first[4], ref.top(_np(x), k))
        return
    h_x = _np(x)
    for k in (0, 4, 32):
        targets = np.full(14, last, np.int32)
        _check_logprob(cs, handle, x, h_x, targets, 1.0, k)
        targets[:] = -1
        _check_logprob(cs, handle, x, h_x, targets, 0.5, k)
    _check_logprob(cs, handle, x, h_x, None, 1.0, 2)


@pytest.mark.parametrize("rows", [2, 700])
def test_token_logprob_alternatives_in_few_hands(cs, handle, rows):
    """All that is not masked lies in the accesses of eight lanes, more of it than the
    list of candidates holds; and the same above a floor of equal logits."""
    vocab = 65536
    at = torch.arange(vocab, device="cuda")
    few = (at // 4 % 32 < 8) & (at // 128 % 32 < 4)
    torch.manual_seed(3)
    for low in (-float("inf"), -7.0):
        x = torch.full((rows, vocab), low, device="cuda")
        x[:, few] = torch.randn(rows, int(few.sum()), device="cuda")
        assert int(few.sum()) > 1024
        _, _, lse, lp, index = cs.token_logprob(handle, x, None, top=32)
        want = torch.topk(x, 32, dim=1)
        assert torch.equal(index.long(), want.indices)
        assert torch.allclose(lp, want.values - lse[:, None], atol=1e-5)


def test_token_logprob_empty(cs, handle):
    x = torch.randn(3, 8, device="cuda")
    t = torch.tensor([0, -1, 2], dtype=torch.int32, device="cuda")
    lp, ent, lse, tl, ti = cs.token_logprob(handle, x[:, :0], t, top=2)
    assert bool((lse == -float("inf")).all()) and not bool(ent.any()) and not bool(lp.any())
    assert bool((ti == -1).all()) and bool((tl == -float("inf")).all())
    assert [o.shape[0] for o in cs.token_logprob(handle, x[:0], t[:0], top=2)] == [0] * 5
    assert cs.token_logprob_grad(handle, x[:0], t[:0], lse[:0], None, lse[:0]).shape == (0, 8)
    assert cs.token_logprob_grad(handle, x[:, :0], t, lse, None, lp).shape == (3, 0)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("rows,vocab,pad,offset", [
    (1, 1, 0, 0), (3, 2, 0, 0), (5, 100, 0, 0), (33, 1001, 0, 0), (7, 4096, 8, 0), (9, 5003, 5, 1),
    (170, 777, 0, 0), (2, 50001, 0, 3), (1, 131072, 0, 0)])
@pytest.mark.parametrize("use", ["both", "logprob", "entropy"])
def test_token_logprob_grad(cs, handle, t, rows, vocab, pad, offset, use):
    rng = np.random.default_rng(rows * 7 + vocab)
    alpha = float(np.float32(1.25))
    x, _ = _make(rng, (rows, vocab), t, 2.0, pad=pad, offset=offset)
    if rows > 4:
        x[1] = -float("inf")                           # nothing left
        x[2, ::2] = -float("inf")
        x[3] = float(torch.finfo(DT[t]).min)
    h_x = _np(x)
    targets = rng.integers(-1, vocab + 1, rows).astype(np.int32)
    targets[0] = vocab - 1
    want, _ = ref.token_logprob(h_x, targets, alpha)
    lse, ent = (torch.from_numpy(want[k]).float().cuda() for k in ("lse", "entropy"))
    up, h_up = _vec(rng, rows, "f32", 0.5, -1.0)
    de, h_de = _vec(rng, rows, "f32", 0.3)
    if use == "logprob":
        de = h_de = None
    if use == "entropy":
        up = h_up = None
    d_t = torch.from_numpy(targets).cuda()
    got = cs.token_logprob_grad(handle, x, d_t, lse, ent, up, de, alpha=alpha)
    v, bound = ref.token_logprob_grad(h_x, targets, _np(lse), _np(ent), h_up, h_de, alpha, t)
    _near(_np(got), v, bound, "dlogits")
    same = cs.token_logprob_grad(handle, x, d_t, lse, ent, up, de, alpha=alpha, out=x)
    assert same.data_ptr() == x.data_ptr() and torch.equal(same, got), "in place"


def test_token_logprob_gradient_against_differences(cs, handle):
    rng = np.random.default_rng(3)
    x, h_x = _make(rng, (4, 11), "f32", 1.5)
    targets = np.array([3, -1, 0, 10], np.int32)
    up, h_up = _vec(rng, 4, "f32")
    de, h_de = _vec(rng, 4, "f32")
    d_t = torch.from_numpy(targets).cuda()
    _, ent, lse = cs.token_logprob(handle, x, d_t, alpha=1.5)
    got = cs.token_logprob_grad(handle, x, d_t, lse, ent, up, de, alpha=1.5)

    def loss(v):
        out, _ = ref.token_logprob(v, targets, 1.5)
        return float((out["logprob"] * h_up + out["entropy"] * h_de).sum())

    _against_differences(loss, h_x, _np(got))


# ---- long buffers, streams, graphs, strides ---------------------------------------

def test_offsets_past_32_bits(cs, handle):
    """Rows whose element offsets pass 2^31, in every matrix."""
    vocab, dim = 1_100_000, 2048                       # 2.25 G elements, 4.5 GB
    table = torch.empty(vocab, dim, dtype=torch.bfloat16, device="cuda")
    table[-3:] = torch.randn(3, dim, device="cuda").bfloat16()
    ids = torch.tensor([vocab - 1, vocab - 3], dtype=torch.int32, device="cuda")
    assert torch.equal(cs.embedding(handle, ids, table), table[[-1, -3]])
    d = torch.randn(2, dim, device="cuda").bfloat16()
    table[-3:] = 0
    cs.embedding_grad(handle, ids, d, table, beta=1.0)
    assert torch.equal(table[[-1, -3]], d)
    big = table.view(-1, 65536)[:, :65521]             # 34375 rows, odd width, long stride
    rows = big.shape[0]
    x = torch.randn(2, 65521, device="cuda").bfloat16()
    big[-2:] = x
    t = torch.full((rows,), 77, dtype=torch.int32, device="cuda")
    part = slice(rows - 2, rows)
    lp, ent, lse, tl, ti = cs.token_logprob(handle, big, t, top=3)
    few = cs.token_logprob(handle, x, t[:2], top=3)
    assert torch.allclose(lp[part], few[0], atol=1e-5) and torch.equal(ti[part], few[4])
    up = torch.ones(rows, device="cuda")
    out = cs.token_logprob_grad(handle, x, t[:2], lse[part].contiguous(), None, up[:2])
    cs.token_logprob_grad(handle, big, t, lse, None, up, out=big)
    assert torch.equal(big[part], out)
    big[-2:] = x
    y, mean, rstd = cs.layer_norm(handle, big, out=big)
    y2, mean2, rstd2 = cs.layer_norm(handle, x)
    assert torch.equal(y[part], y2) and torch.equal(mean[part], mean2)


def test_another_stream_and_graph_capture(cs):
    """The whole chain on a side stream, then captured in a graph after a reserve."""
    torch.manual_seed(1)
    vocab, dim, n = 500, 136, 300
    table = torch.randn(vocab, dim, device="cuda")
    head = torch.randn(dim, vocab, device="cuda")
    ids = torch.randint(0, vocab, (n,), device="cuda", dtype=torch.int32)
    w, b = torch.rand(dim, device="cuda"), torch.rand(dim, device="cuda")
    with cs.Handle(0) as h:
        h.reserve_lm(n, dim)

        def chain(stream):
            x = cs.embedding(h, ids, table, scale=2.0, stream=stream)
            y, mean, rstd = cs.layer_norm(h, x, w, b, stream=stream)
            z = y @ head
            lp, ent, lse = cs.token_logprob(h, z, ids, stream=stream)
            dz = cs.token_logprob_grad(h, z, ids, lse, ent, -torch.ones_like(lp),
                                       stream=stream)
            dx, dw, db = cs.layer_norm_grad(h, dz @ head.T, x, mean, rstd, w, stream=stream)
            dt = torch.empty_like(table)
            cs.embedding_grad(h, ids, dx, dt, scale=2.0, stream=stream)
            return lp, dw, db, dt

        want = chain(None)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = chain(side)
        side.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, got))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = chain(None)
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(want, held))


def test_c_refusals(cs, handle):
    """What the C entry points refuse on a live handle, before any launch."""
    inv, dim_, null = (cs.SPMM_ERR_INVALID_ARGUMENT, cs.SPMM_ERR_DIMENSION_MISMATCH,
                       cs.SPMM_ERR_NULL_POINTER)
    h, x = handle.ptr, torch.zeros(64, device="cuda")
    a = x.data_ptr()
    i = torch.zeros(64, dtype=torch.int32, device="cuda").data_ptr()

    def status(fn, *args):
        return fn(h, *args, check=False)

    E, G = cs.spmm_embedding, cs.spmm_embedding_grad
    assert status(E, 3, 1.0, i, 2, a, 4, 4, 4, a, 4) == inv
    assert status(E, 0, 1.0, i, -1, a, 4, 4, 4, a, 4) == inv
    assert status(E, 0, 1.0, i, 2, a, 3, 4, 4, a, 4) == dim_
    assert status(E, 0, 1.0, i, 2, a, 4, 4, 4, a, 3) == dim_
    assert status(E, 0, 1.0, 0, 2, a, 4, 4, 4, a, 4) == null
    assert status(E, 0, 1.0, i, 2, 0, 4, 4, 4, a, 4) == null
    assert status(G, 1, 2, 1.0, i, 2, a, 4, 0.0, a, 4, 4, 4) == inv
    assert status(G, 0, 0, 1.0, i, (1 << 30) + 1, a, 4, 0.0, a, 4, 4, 4) == inv
    assert status(G, 0, 0, 1.0, i, 2, a, 3, 0.0, a, 4, 4, 4) == dim_
    assert status(G, 0, 0, 1.0, i, 2, 0, 4, 0.0, a, 4, 4, 4) == null
    N, D = cs.spmm_layer_norm, cs.spmm_layer_norm_grad
    assert status(N, 0, 0, a, 4, 2, 4, 0, 0, -1.0, a, 4, 0, 0) == inv
    assert status(N, 0, 0, a, 4, 2, 4, 0, 0, float("nan"), a, 4, 0, 0) == inv
    assert status(N, 0, 1, a, 4, 2, 4, 0, 0, 0.0, a, 4, 0, 0) == inv
    assert status(N, 0, 0, a, 3, 2, 4, 0, 0, 0.0, a, 4, 0, 0) == dim_
    assert status(N, 0, 0, 0, 4, 2, 4, 0, 0, 0.0, a, 4, 0, 0) == null
    assert status(D, 0, 0, a, 4, a, 4, a, a, 0, 2, 4, a, 3, 0, 0) == dim_
    assert status(D, 0, 0, a, 4, a, 4, 0, a, 0, 2, 4, a, 4, 0, 0) == null
    P, Q = cs.spmm_token_logprob, cs.spmm_token_logprob_grad
    for alpha in (0.0, -1.0, float("inf"), float("nan")):
        assert status(P, 0, alpha, a, 4, 2, 4, i, 0, a, a, a, 0, 0) == inv
        assert status(Q, 0, alpha, a, 4, 2, 4, i, a, a, a, a, a, 4) == inv
    for k in (-1, 33):
        assert status(P, 0, 1.0, a, 4, 2, 4, i, k, a, a, a, a, i) == inv
    assert status(P, 0, 1.0, a, 3, 2, 4, i, 0, a, a, a, 0, 0) == dim_
    assert status(P, 0, 1.0, a, 4, 2, 4, i, 0, 0, a, a, 0, 0) == null
    assert status(P, 0, 1.0, a, 4, 2, 4, i, 2, a, a, a, a, 0) == null
    assert status(Q, 0, 1.0, a, 4, 2, 4, i, a, a, a, a, a, 3) == dim_
    assert status(Q, 0, 1.0, a, 4, 2, 4, 0, a, a, a, a, a, 4) == null
    assert status(Q, 0, 1.0, a, 4, 2, 4, i, a, 0, a, a, a, 4) == null
    assert status(Q, 0, 1.0, a, 4, 2, 4, i, 0, a, a, a, a, 4) == null
    for call in (lambda: cs.embedding(handle, torch.zeros(2, dtype=torch.int32, device="cuda"),
                                      torch.zeros(1, 4, device="cuda").expand(3, 4)),
                 lambda: cs.layer_norm(handle, torch.zeros(1, 4, device="cuda").expand(3, 4))):
        with pytest.raises(cs.SpmmError) as e:        # rows that overlap
            call()
        assert e.value.status == dim_
    assert not bool(x.any())
