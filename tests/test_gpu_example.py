"""The example model trains: its loss falls from the uniform one, and its gradients (through
every operator of the step) agree with torch's own."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import __graft_entry__
    __graft_entry__.build_library()
    spec = importlib.util.spec_from_file_location(
        "token_mixing_lm", os.path.join(ROOT, "examples", "token_mixing_lm.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_loss_falls(example):
    losses = example.main(["--quiet"])
    assert abs(losses[0] - math.log(200)) < 1.5
    assert losses[-1] < 0.2 * losses[0]


def test_one_step_against_autograd(example):
    """A step of size 1 moves each parameter by minus its gradient."""
    import csr_spmm_gb300 as cs
    n, vocab, dim, window = 300, 50, 24, 3
    model = example.Model(vocab, dim, seed=4)
    gen = torch.Generator(device="cuda").manual_seed(2)
    ids, targets = (torch.randint(0, vocab, (n,), generator=gen, device="cuda", dtype=torch.int32)
                    for _ in range(2))
    mix, mix_t = example.band(n, window)
    params = [p.clone().double().requires_grad_() for p in (model.table, model.weight,
                                                              model.bias)]
    table, weight, bias = params
    a = torch.zeros(n, n, dtype=torch.float64, device="cuda")
    for t in range(n):
        first = max(0, t - window + 1)
        a[t, first:t + 1] = 1.0 / (t + 1 - first)
    h = torch.nn.functional.layer_norm(a @ (math.sqrt(dim) * table[ids.long()]), (dim,), weight,
                                       bias)
    loss = torch.nn.functional.cross_entropy(h @ table.T, targets.long())
    loss.backward()
    before = [p.detach() for p in params]
    with cs.Handle(0) as handle:
        got = model.step(handle, ids, targets, mix, mix_t, rate=1.0)
    assert abs(float(got) - float(loss.detach())) < 1e-5
    for old, new, p in zip(before, (model.table, model.weight, model.bias), params):
        # binary32 throughout: sums of at most a few thousand terms, matrix products included
        assert torch.allclose(old - new.double(), p.grad, atol=2e-5 * float(p.grad.abs().max()) + 1e-6)
