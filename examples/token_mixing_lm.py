"""A small language model on this library's operators, trained on a repeating text.

    python examples/token_mixing_lm.py [--steps N]

A token's state is the normalised mean, over the last `window` tokens, of their
embeddings; the next token's logits are its products with the embeddings (the
table is tied).  One training step is

    x  = embedding(ids)                    scaled lookup
    m  = A x                               spmm, A the banded CSR matrix of the means
    h  = layer_norm(m)
    z  = h E^T                             a plain matrix product
    lp = token_logprob(z)                  log probability of each next token
    dz = token_logprob_grad(...)
    dE = dz^T h                            a plain matrix product
    dm = layer_norm_grad(dz E)
    dx = A^T dm                            spmm with the transposed matrix
    dE += embedding_grad(dx)               beta = 1: added to what dE holds

followed by a step of gradient descent.  Everything runs in binary32 on one GPU.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import csr_spmm_gb300 as cs  # noqa: E402


def band(n: int, window: int):
    """CSR arrays of the n x n matrix whose row t averages tokens t - window + 1 .. t,
    and of its transpose."""
    rows = np.repeat(np.arange(n), window)
    cols = rows - np.tile(np.arange(window)[::-1], n)
    keep = cols >= 0
    rows, cols = rows[keep], cols[keep]
    count = np.minimum(np.arange(n) + 1, window)
    vals = (1.0 / count)[rows].astype(np.float32)

    def csr(r, c, v):
        order = np.lexsort((c, r))
        ptr = np.zeros(n + 1, np.int32)
        np.cumsum(np.bincount(r, minlength=n), out=ptr[1:])
        return tuple(torch.from_numpy(a).cuda() for a in (ptr, c[order].astype(np.int32),
                                                          v[order]))

    return csr(rows, cols, vals), csr(cols, rows, vals)


class Model:
    def __init__(self, vocab: int, dim: int, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.table = 0.1 * torch.randn(vocab, dim, generator=gen, device="cuda")
        self.weight = torch.ones(dim, device="cuda")
        self.bias = torch.zeros(dim, device="cuda")
        self.scale = math.sqrt(dim)

    def step(self, handle, ids, targets, mix, mix_t, rate: float) -> torch.Tensor:
        """One step of gradient descent; returns the mean loss (on the device)."""
        n, dim = ids.numel(), self.table.shape[1]
        x = cs.embedding(handle, ids, self.table, scale=self.scale)
        m = torch.empty_like(x)
        cs.spmm(handle, 1.0, *mix, n, x, 0.0, m)
        h, mean, rstd = cs.layer_norm(handle, m, self.weight, self.bias)
        z = h @ self.table.T
        logprob, _, lse = cs.token_logprob(handle, z, targets)
        loss = -logprob.mean()

        up = torch.full((n,), -1.0 / n, device="cuda")
        dz = cs.token_logprob_grad(handle, z, targets, lse, dlogprob=up, out=z)
        dtable = dz.T @ h
        dm, dweight, dbias = cs.layer_norm_grad(handle, dz @ self.table, m, mean, rstd,
                                                self.weight)
        dx = torch.empty_like(x)
        cs.spmm(handle, 1.0, *mix_t, n, dm, 0.0, dx)
        cs.embedding_grad(handle, ids, dx, dtable, scale=self.scale, beta=1.0)
        for value, grad in ((self.table, dtable), (self.weight, dweight), (self.bias, dbias)):
            value.sub_(grad, alpha=rate)
        return loss

    def alternatives(self, handle, ids, mix, top: int):
        """The most likely next tokens after `ids` and their log probabilities."""
        x = cs.embedding(handle, ids, self.table, scale=self.scale)
        m = torch.empty_like(x)
        cs.spmm(handle, 1.0, *mix, ids.numel(), x, 0.0, m)
        h, _, _ = cs.layer_norm(handle, m, self.weight, self.bias)
        _, _, _, logprob, index = cs.token_logprob(handle, h[-1:] @ self.table.T, top=top)
        return index[0].tolist(), logprob[0].tolist()


def main(argv=None) -> list:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--quiet", action="store_true")
    a = ap.parse_args(argv)
    vocab, dim, window, n = 200, 64, 2, 2000
    text = np.random.default_rng(1).permutation(vocab).astype(np.int32)   # its period
    ids = torch.from_numpy(np.resize(text, n)).cuda()
    targets = torch.from_numpy(np.resize(np.roll(text, -1), n)).cuda()
    mix, mix_t = band(n, window)
    model, losses = Model(vocab, dim), []
    with cs.Handle(0) as handle:
        for i in range(a.steps):
            loss = float(model.step(handle, ids, targets, mix, mix_t, rate=2.0))
            losses.append(loss)
            if not a.quiet and i % 20 == 0:
                print(f"step {i:3d}  loss {loss:.4f}")
        m = 20
        short, _ = band(m, window)
        index, logprob = model.alternatives(handle, ids[:m], short, 3)
    if not a.quiet:
        print(f"last loss {losses[-1]:.4f} (uniform: {math.log(vocab):.4f})")
        print(f"after token {int(ids[m - 1])} comes {int(targets[m - 1])}; most likely: "
              + ", ".join(f"{i} ({math.exp(p):.3f})" for i, p in zip(index, logprob)))
    return losses


if __name__ == "__main__":
    main()
