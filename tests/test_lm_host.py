"""The language-model operators' argument checks, on the host (no GPU)."""
import types

import pytest

import csr_spmm_gb300 as cs
from csr_spmm_gb300 import _lib

torch = pytest.importorskip("torch")

FAKE = types.SimpleNamespace(ptr=None, device=0)       # never reaches the library
F = torch.zeros
IDS = torch.zeros(3, dtype=torch.int32)


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.library()


def test_null_handles_are_refused_before_any_device_work(lib):
    inv = cs.SPMM_ERR_INVALID_ARGUMENT
    assert lib.spmm_reserve_lm(None, 4, 4) == inv
    assert lib.spmm_embedding(None, 0, 1.0, None, 4, None, 4, 4, 4, None, 4, None) == inv
    assert lib.spmm_embedding_grad(None, 0, 0, 1.0, None, 4, None, 4, 0.0, None, 4, 4, 4,
                                   None) == inv
    assert lib.spmm_layer_norm(None, 0, 0, None, 4, 4, 4, None, None, 0.0, None, 4, None, None,
                               None) == inv
    assert lib.spmm_layer_norm_grad(None, 0, 0, None, 4, None, 4, None, None, None, 4, 4, None, 4,
                                    None, None, None) == inv
    assert lib.spmm_token_logprob(None, 0, 1.0, None, 4, 4, 4, None, 0, None, None, None, None,
                                  None, None) == inv
    assert lib.spmm_token_logprob_grad(None, 0, 1.0, None, 4, 4, 4, None, None, None, None, None,
                                       None, 4, None) == inv


def _calls():
    """One call of each operator, by name, on the given tensors."""
    return {
        "embedding": lambda **k: cs.embedding(FAKE, k.get("ids", IDS), k.get("table", F(5, 8)),
                                              out=k.get("out")),
        "embedding_grad": lambda **k: cs.embedding_grad(
            FAKE, k.get("ids", IDS), k.get("dout", F(3, 8)), k.get("dtable", F(5, 8))),
        "layer_norm": lambda **k: cs.layer_norm(FAKE, k.get("x", F(3, 8)), k.get("weight", F(8)),
                                                k.get("bias", F(8)), out=k.get("out")),
        "layer_norm_grad": lambda **k: cs.layer_norm_grad(
            FAKE, k.get("dy", F(3, 8)), k.get("x", F(3, 8)), k.get("mean", F(3)),
            k.get("rstd", F(3)), k.get("weight", F(8)), out=k.get("out")),
        "token_logprob": lambda **k: cs.token_logprob(
            FAKE, k.get("logits", F(3, 8)), k.get("targets", IDS), top=k.get("top", 0)),
        "token_logprob_grad": lambda **k: cs.token_logprob_grad(
            FAKE, k.get("logits", F(3, 8)), k.get("targets", IDS), k.get("lse", F(3)),
            k.get("entropy", F(3)), k.get("dlogprob", F(3)), k.get("dentropy", F(3)),
            out=k.get("out")),
    }


@pytest.mark.parametrize("op", sorted(_calls()))
def test_host_tensors_are_refused(op):
    with pytest.raises(ValueError, match="CUDA tensor"):
        _calls()[op]()


@pytest.mark.parametrize("op,what,error,match", [
    ("embedding", dict(ids=IDS.long()), TypeError, "ids must be int32"),
    ("embedding", dict(ids=torch.zeros(6, dtype=torch.int32)[::2]), ValueError, "contiguous"),
    ("embedding", dict(ids=torch.zeros(1, 3, dtype=torch.int32)), ValueError, "1-D"),
    ("embedding", dict(table=F(5, 8).double()), TypeError, "float32, float16 or bfloat16"),
    ("embedding", dict(table=F(8, 5).t()), ValueError, "unit column stride"),
    ("embedding", dict(table=F(40)), ValueError, "2-D"),
    ("embedding", dict(out=F(3, 9)), ValueError, "out must be"),
    ("embedding", dict(out=F(3, 8).half()), TypeError, "out must be float32"),
    ("embedding_grad", dict(dtable=F(5, 9)), ValueError, "shape mismatch"),
    ("embedding_grad", dict(dtable=F(5, 8).half()), TypeError, "dout's dtype"),
    ("embedding_grad", dict(dout=F(4, 8)), ValueError, "4 entries"),
    ("layer_norm", dict(weight=F(7)), ValueError, "8 entries"),
    ("layer_norm", dict(weight=F(8).half()), TypeError, "x's dtype"),
    ("layer_norm", dict(x=F(3, 8).half(), weight=F(8), bias=F(8).half()), TypeError,
     "bias must be float32"),
    ("layer_norm", dict(bias=F(16)[::2]), ValueError, "contiguous"),
    ("layer_norm", dict(x=F(8, 3).t()), ValueError, "unit column stride"),
    ("layer_norm_grad", dict(dy=F(3, 7)), ValueError, "shape mismatch"),
    ("layer_norm_grad", dict(dy=F(3, 8).half()), TypeError, "one dtype"),
    ("layer_norm_grad", dict(mean=F(2)), ValueError, "3 entries"),
    ("layer_norm_grad", dict(rstd=F(3).double()), TypeError, "rstd must be float32"),
    ("layer_norm_grad", dict(out=F(2, 8)), ValueError, "out must be"),
    ("token_logprob", dict(targets=IDS[:2]), ValueError, "3 entries"),
    ("token_logprob", dict(targets=IDS.long()), TypeError, "targets must be int32"),
    ("token_logprob", dict(top=33), ValueError, "top must be"),
    ("token_logprob", dict(top=-1), ValueError, "top must be"),
    ("token_logprob_grad", dict(targets=None), ValueError, "needs the targets"),
    ("token_logprob_grad", dict(entropy=None), ValueError, "needs the entropy"),
    ("token_logprob_grad", dict(lse=F(4)), ValueError, "3 entries"),
    ("token_logprob_grad", dict(dlogprob=F(3).half()), TypeError, "dlogprob must be float32"),
    ("token_logprob_grad", dict(out=F(3, 9)), ValueError, "out must be"),
])
def test_refusals(op, what, error, match):
    with pytest.raises(error, match=match):
        _calls()[op](**what)


class _AsCuda(torch.Tensor):
    """A host tensor that reports itself as on cuda:0."""

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", 0)

    def get_device(self):
        return 0


def _cuda(t):
    return torch.Tensor._make_subclass(_AsCuda, t)


def test_calls_pass_addresses_and_leading_dimensions(monkeypatch):
    calls = []
    for name in ("spmm_embedding", "spmm_embedding_grad", "spmm_layer_norm",
                 "spmm_layer_norm_grad", "spmm_token_logprob", "spmm_token_logprob_grad"):
        monkeypatch.setattr(_lib, name, lambda *a, name=name: calls.append((name, a)))
    monkeypatch.setattr(cs.lm, "_current", lambda device: 77)
    h = types.SimpleNamespace(ptr=1234, device=0)
    ids, table, out = _cuda(IDS.clone()), _cuda(F(5, 10))[:, :8], _cuda(F(3, 12))[:, :8]
    assert cs.embedding(h, ids, table, scale=2.0, out=out) is out
    assert calls.pop() == ("spmm_embedding", (1234, 0, 2.0, ids.data_ptr(), 3, table.data_ptr(),
                                              10, 5, 8, out.data_ptr(), 12, 77))
    d16 = _cuda(F(3, 9).bfloat16())[:, :8]
    cs.embedding_grad(h, ids, d16, table, scale=2.0, beta=1.0)
    assert calls.pop() == ("spmm_embedding_grad", (1234, 2, 0, 2.0, ids.data_ptr(), 3,
                                                   d16.data_ptr(), 9, 1.0, table.data_ptr(), 10,
                                                   5, 8, 77))
    logits, lse = _cuda(F(3, 11).half())[:, :8], _cuda(F(3))
    res = _cuda(F(3, 8).half())
    cs.token_logprob_grad(h, logits, ids, lse, None, lse, out=res, alpha=0.5)
    assert calls.pop() == ("spmm_token_logprob_grad", (1234, 1, 0.5, logits.data_ptr(), 11, 3, 8,
                                                       ids.data_ptr(), lse.data_ptr(), 0,
                                                       lse.data_ptr(), 0, res.data_ptr(), 8, 77))
    with pytest.raises(ValueError, match="handle is on cuda:1"):
        cs.embedding(types.SimpleNamespace(ptr=1, device=1), ids, table, out=out)
    assert calls == []


def test_compiled_calls_convert_their_arguments(lib):
    """The raw functions: numbers and addresses as the C signature has them, or an error."""
    inv = cs.SPMM_ERR_INVALID_ARGUMENT
    assert _lib.spmm_embedding(None, 0, 1, 0, 4, None, 4, 4, 4, 0, 4, 0, check=False) == inv
    with pytest.raises(cs.SpmmError, match="spmm_layer_norm"):
        _lib.spmm_layer_norm(None, 0, 0, 0, 4, 4, 4, 0, 0, 0.0, 0, 4, 0, 0)
    calls = _lib.load_module("_lm_calls")
    with pytest.raises(TypeError, match="12 arguments"):
        calls.spmm_embedding(0)
    with pytest.raises(TypeError):
        _lib.spmm_embedding("h", 0, 1.0, 0, 4, 0, 4, 4, 4, 0, 4)
    with pytest.raises(TypeError):
        _lib.spmm_embedding(0, 0, "1.0", 0, 4, 0, 4, 4, 4, 0, 4)
    with pytest.raises(OverflowError):
        _lib.spmm_embedding(0, 0, 1.0, 0, 1 << 63, 0, 4, 4, 4, 0, 4)
    with pytest.raises(ImportError, match="is missing"):
        _lib.load_module("_no_such_module")


def test_outputs_are_refused_in_other_forms(lib):
    new = _lib.load_module("_torch_outputs").new
    with pytest.raises(TypeError, match="type, rows, columns"):
        new(0, 0, 4)
    assert new(0) == ()
    with pytest.raises(ValueError, match="no such type"):
        new(0, 4, 1, 1)
    with pytest.raises(TypeError):
        new(0, 0, "1", 1)


def test_the_package_imports_without_torch():
    """torch is needed by the tensor wrappers only, and loaded on their first use."""
    import subprocess
    import sys
    code = ("import sys; import csr_spmm_gb300 as cs; assert 'torch' not in sys.modules; "
            "cs.SPMM_BF16; from csr_spmm_gb300 import embedding; assert 'torch' in sys.modules; "
            "assert cs.embedding is embedding is cs.lm.embedding; "
            "missing = False\ntry:\n    cs.nothing\nexcept AttributeError:\n    missing = True\n"
            "assert missing")
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
