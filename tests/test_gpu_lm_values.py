"""The language-model operators at the ends of their arguments' ranges: logits that the
inverse temperature takes beyond binary32, and rows that hardly vary."""
import numpy as np
import pytest

import lm_reference as ref
from test_gpu_lm import DT, TYPES, _near, _np, cs, handle  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

INF = float("inf")
LARGEST = float(np.finfo(np.float32).max)


def _counted(x, alpha):
    """The logits as z = alpha x in binary32 counts them: infinite where z is."""
    with np.errstate(over="ignore"):
        z = (np.float32(alpha) * x.astype(np.float32)).astype(np.float64)
    return np.where(np.isinf(z), z, x)


def _stored(value):
    """A result as a binary32 output holds it: infinite beyond the range."""
    return np.where(np.abs(value) > LARGEST, np.copysign(np.inf, value), value)


def _check(cs, handle, x, targets, alpha, k):
    """Against the definition over the counted logits; alternatives in the order of the
    logits themselves."""
    h_x = _np(x)
    c_x = _counted(h_x, alpha)
    a32 = float(np.float32(alpha))
    want, tol = ref.token_logprob(c_x, targets, a32)
    got = cs.token_logprob(handle, x, torch.from_numpy(targets).cuda(), alpha=alpha, top=k)
    for g, name in zip(got[:3], ("logprob", "entropy", "lse")):
        _near(_np(g), _stored(want[name]), tol[name], name)
    if k:
        index = ref.top(np.where(np.isneginf(c_x), c_x, h_x), k)
        assert np.array_equal(got[4].cpu().numpy(), index), "top_index"
        picked = np.take_along_axis(h_x, np.maximum(index, 0), 1)
        lse = want["lse"][:, None]
        with np.errstate(invalid="ignore"):
            lp = np.where(np.isnan(lse), np.nan, np.where(index >= 0, a32 * picked - lse, -np.inf))
            bound = tol["lse"][:, None] + ref.U * (2 * np.abs(a32 * picked) + np.abs(lp))
        _near(_np(got[3]), _stored(lp), bound, "top_logprob")
    up = torch.full((x.shape[0],), -1.0, device="cuda")
    grad = cs.token_logprob_grad(handle, x, torch.from_numpy(targets).cuda(), got[2], got[1], up,
                                 up, alpha=1.0 if alpha > 1e30 else alpha)
    lse = want["lse"]
    assert bool(grad[torch.from_numpy(np.isnan(lse)).cuda()].isnan().all()), "NaN rows"
    assert not bool(grad[torch.from_numpy(np.isneginf(lse)).cuda()].any()), "empty rows"


@pytest.mark.parametrize("times", [1, 90])
@pytest.mark.parametrize("vocab", [9, 1001, 40001])
@pytest.mark.parametrize("t,alpha", [("f32", 1.25), ("f32", 2.0), ("bf16", 1.25), ("bf16", 3.0),
                                     ("f16", 7e33)])
def test_logits_that_alpha_takes_beyond_binary32(cs, handle, t, alpha, vocab, times):  # noqa: F811
    """They count as infinite ones: below, masked; above, the row is NaN."""
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy(rng.standard_normal((10, vocab)) * 2).to(DT[t]).cuda()
    low, high = float(torch.finfo(DT[t]).min), float(torch.finfo(DT[t]).max)
    last = vocab - 1
    x[0] = low                                         # masked throughout
    x[1] = high
    x[2] = low
    x[2, vocab // 2] = 0.5                             # one left
    x[3, vocab // 3] = high
    x[4, last] = low                                   # the target is masked
    x[5] = low
    x[5, 1] = float("nan")
    x[6] = -INF
    x[6, 2] = low
    x[7] = low                                         # the largest is just within the range
    x[7, 4] = -0.9 * LARGEST / alpha
    x[8] = 0.9 * LARGEST / alpha
    targets = np.full(10, last, np.int32)
    if times > 1:
        x, targets = x.repeat(times, 1), np.tile(targets, times)
    for k in (0, 5):
        _check(cs, handle, x, targets, alpha, k)
    targets[:] = -1
    _check(cs, handle, x, targets, alpha, 0)


@pytest.mark.parametrize("rows", [7, 700])
def test_the_largest_alpha(cs, handle, rows):  # noqa: F811
    """alpha times log2(e) is beyond binary32 too: only logits near zero are within it."""
    x = torch.full((rows, 50), -1.0, device="cuda")
    x[0, [3, 9]] = 0.0                                 # z = 0 twice
    x[1, 5] = 1e-38                                    # z = 3, and 0 beside it
    x[1, 7] = 0.0
    x[3, 8] = 1.0                                      # beyond the range
    x[4, 2] = -0.5
    x[5, 30:] = 0.0
    _check(cs, handle, x, np.full(rows, 7, np.int32), 3e38, 4)


@pytest.mark.parametrize("rows", [6, 900])
@pytest.mark.parametrize("dim", [1, 3, 7, 100, 515, 768, 1000, 2500, 4096, 5000, 8200, 16384,
                                 20001, 40960])
@pytest.mark.parametrize("t", TYPES)
def test_layer_norm_of_constant_rows(cs, handle, t, dim, rows):  # noqa: F811
    """A constant row's mean is the constant, so its deviations are 0: y is the bias, rstd is
    1 / sqrt(eps), and eps == 0 gives 0 * inf."""
    if rows > 100 and dim > 9000:
        rows = 310
    values = torch.tensor([1000.0, 0.1, -3.3, 60001.7, 1.0 / 3.0, -0.0077], device="cuda")
    c = values.repeat(-(-rows // 6))[:rows].to(DT[t])
    x = c[:, None].expand(rows, dim).contiguous()
    w = torch.linspace(0.5, 2.0, dim, device="cuda").to(DT[t])
    b = torch.linspace(-1.0, 1.0, dim, device="cuda").to(DT[t])
    layouts = [x]
    if dim < 9000:
        off = torch.empty(rows * dim + 1, dtype=DT[t], device="cuda")[1:].view(rows, dim)
        layouts.append(off.copy_(x))                   # rows between 16-byte boundaries
    for rows_of in layouts:
        y, mean, rstd = cs.layer_norm(handle, rows_of, w, b, eps=1e-5)
        assert torch.equal(mean, c.float())
        assert torch.equal(y, b.expand(rows, dim))
        want = 1.0 / np.sqrt(float(np.float32(1e-5)))
        assert bool(((rstd.double() - want).abs() <= 6 * ref.U * want).all())
        y, _, rstd = cs.layer_norm(handle, rows_of, eps=0.0)
        assert bool(y.isnan().all()) and bool(rstd.isinf().all())


@pytest.mark.parametrize("rows", [5, 700])
@pytest.mark.parametrize("dim", [64, 1001, 4096, 16384, 20001])
def test_layer_norm_of_rows_that_hardly_vary(cs, handle, dim, rows):  # noqa: F811
    """Binary32 rows whose deviations are a few units of their last place: all that the mean's
    own rounding (half a unit) leaves is held to, far below the sums' roundings."""
    if rows > 100 and dim > 9000:
        rows = 310
    rng = np.random.default_rng(dim)
    ulp = 2.0 ** -14                                   # of numbers in [512, 1024)
    h_x = 700.0 + ulp * rng.integers(-20, 21, (rows, dim))
    x = torch.from_numpy(h_x).float().cuda()
    assert np.array_equal(_np(x), h_x)
    y, mean, rstd = cs.layer_norm(handle, x, eps=0.0)
    m = h_x.mean(1, keepdims=True)
    dev = h_x - m
    r = 1.0 / np.sqrt((dev * dev).mean(1, keepdims=True))
    # the mean is off by half a unit for its rounding; what corrects it is a sum of deviations
    # of at most 200 units (the first mean's error and 20), off by its chain of about 180 U of
    # that: under 1/64 of a unit
    d_mean = ulp * (0.5 + 1 / 64)
    _near(_np(mean), m[:, 0], d_mean, "mean")
    d_rstd = r * (0.5 * d_mean ** 2 * r ** 2 + ref.U * (ref.chain(dim) + 12))
    _near(_np(rstd), r[:, 0], d_rstd[:, 0], "rstd")
    _near(_np(y), dev * r, d_mean * (r + d_rstd) + np.abs(dev) * d_rstd + 4 * ref.U * np.abs(dev * r),
          "y")


@pytest.mark.parametrize("rows", [5, 400])
@pytest.mark.parametrize("dim", [64, 444, 600, 2276, 2277, 5312, 8200])
@pytest.mark.parametrize("t", TYPES)
def test_layer_norm_of_rows_with_outliers(cs, handle, t, dim, rows):  # noqa: F811
    """Columns of large values, where rows and parts of rows begin among them: neither the mean
    nor the deviations lose digits to them."""
    rng = np.random.default_rng(dim + rows)
    for columns in (slice(0, 1), slice(None, None, 512), slice(None, None, dim // 3 + 1)):
        x = torch.from_numpy(rng.standard_normal((rows, dim)) * 1.5 + 0.25).to(DT[t])
        x[:, columns] *= 60
        y, mean, rstd = cs.layer_norm(handle, x.cuda(), eps=1e-3)
        want = ref.layer_norm(x.double().numpy(), 1.0, 0.0, float(np.float32(1e-3)), t)
        for g, (v, bound), what in zip((y, mean, rstd), want, ("y", "mean", "rstd")):
            _near(_np(g), v, bound, what)


@pytest.mark.parametrize("rows", [7, 700])
@pytest.mark.parametrize("vocab", [100, 5003])
@pytest.mark.parametrize("t,alpha", [("f32", 0.7), ("f32", 1.25), ("f32", 0.3), ("bf16", 0.7),
                                     ("bf16", 1.1), ("f16", 0.7), ("f16", 900.7)])
def test_logits_whose_last_place_is_larger_than_their_differences(cs, handle, t, alpha, vocab,  # noqa: F811
                                                                  rows):
    """Rows of equal logits of large magnitude (a type's lowest values as masks throughout): z and
    lse are binary32 numbers some of whose places are lost, but lost alike: no log probability
    is above 0 or below by more than a place, and the gradient is the formula's of those numbers."""
    low, high = float(torch.finfo(DT[t]).min), float(torch.finfo(DT[t]).max)
    values = torch.tensor([low / 4, high / 8, low / 3, -6.1e4, 5.3e4, low / 1000, 777.0],
                          device="cuda").to(DT[t])
    x = values.repeat(rows // 7)[:, None].expand(rows, vocab).contiguous()
    x[:, 3] = -INF
    targets = torch.full((rows,), vocab - 1, dtype=torch.int32, device="cuda")
    lp, ent, lse, best, index = cs.token_logprob(handle, x, targets, alpha=alpha, top=2)
    z = np.float32(alpha) * _np(x[:, -1]).astype(np.float32)
    assert z.dtype == np.float32 and np.isfinite(z).all()
    place = np.spacing(np.abs(z)).astype(np.float64)
    n = vocab - 1
    # lse and z are rounded once each, log(n) beside them; their difference once more
    bound = 1.01 * place + ref.U * (ref.chain(vocab) + 16) * (1 + np.log(n))
    _near(_np(lse), z.astype(np.float64) + np.log(n), bound, "lse")
    _near(_np(lp), np.full(rows, -np.log(n)), bound + place / 2, "logprob")
    assert bool((lp <= 0).all()) and torch.equal(best, lp[:, None].expand(rows, 2))
    assert index.tolist() == [[0, 1]] * rows
    _near(_np(ent), np.full(rows, np.log(n)), ref.U * (ref.chain(vocab) + 24) * np.log(n), "entropy")
    up = torch.full((rows,), -1.0, device="cuda")
    got = cs.token_logprob_grad(handle, x, targets, lse, ent, up, 0.5 * up, alpha=alpha)
    a32 = float(np.float32(alpha))
    # below 2^20, z - lse is taken in one rounding
    exact = a32 * _np(x[:, -1])
    q = np.where(np.abs(_np(lse)) < 2.0 ** 20, exact, z.astype(np.float64)) - _np(lse)
    p = np.exp(q)
    want = np.zeros((rows, vocab))
    want += (a32 * p * (1 + 0.5 * (q + _np(ent))))[:, None]
    want[:, -1] -= a32
    want[:, 3] = 0.0
    # the exponential is off by 8 U and its argument by 2 U of itself; the terms by their roundings
    scale = a32 * (p * (1 + np.abs(q) + np.abs(_np(ent))) + 1)[:, None]
    _near(_np(got), want, 40 * ref.U * (1 + np.abs(q))[:, None] * scale + ref.rounding(t, want),
          "dlogits")


@pytest.mark.parametrize("rows", [3, 350])
@pytest.mark.parametrize("dim", [5, 64, 1001, 4096, 20001])
def test_layer_norm_beyond_the_range_of_squares(cs, handle, dim, rows):  # noqa: F811
    """Deviations whose squares overflow have rstd 0, so y is the bias; an infinite element makes
    the row NaN."""
    x = torch.randn(rows, dim, device="cuda") * 1e25
    x[:, 0] = 3e25
    w = torch.linspace(0.5, 2.0, dim, device="cuda")
    b = torch.linspace(-1.0, 1.0, dim, device="cuda")
    y, mean, rstd = cs.layer_norm(handle, x, w, b)
    assert not bool(rstd.any()) and torch.equal(y, b.expand(rows, dim))
    assert bool(((mean.double() - x.double().mean(1)).abs() < 1e21).all())
    x[1, dim // 2] = INF
    x[2, dim - 1] = -INF
    y, mean, rstd = cs.layer_norm(handle, x, w, b)
    assert bool(y[1:3].isnan().all()) and bool(rstd[1:3].isnan().all())
    assert torch.equal(y[0], b)
