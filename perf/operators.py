"""The two ends of a language model on the GPU: the operators, their cases and their plain forms.

Six operators, three pairs of a forward pass and its gradient:

* ``embedding`` / ``embedding_grad``: ``out[t] = scale * table[ids[t]]`` and its gradient, the
  product of the transposed one-entry-per-row matrix with the gradient of ``out``;
* ``layer_norm`` / ``layer_norm_grad``: normalisation of each row, and the gradients of the row,
  the weight and the bias;
* ``token_logprob`` / ``token_logprob_grad``: from a matrix of logits, each row's log probability
  of a given token, its entropy, log-sum-exp and top alternatives; and the logits' gradient.

Where ``own`` is false, ``run`` computes them in elementary torch operations in 32 bits; where it
is true, it calls this package's operators.  ``exact`` computes the definitions in 64 bits.

Conventions that both follow: an id (or target) outside [0, vocabulary) is padding: its embedding
row is zero, it takes no part in any gradient of a log probability, and its log probability is 0.
A logit of -inf is masked: it has probability 0 and is never an alternative; an alternative that
does not exist has index -1 and log probability -inf.  Equal logits rank by lowest index.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5


def listed():
    return [
        # one step of generation for 16 sequences: one id each, a few rows of the table
        {"name": "embed_decode", "op": "embedding", "type": "bf16", "tokens": 16, "vocab": 32768,
         "dim": 2048, "pad": 0.0},
        # the prompts of a large batch, padded to one length: a gigabyte of rows
        {"name": "embed_prompts", "op": "embedding", "type": "bf16", "tokens": 100003,
         "vocab": 131072, "dim": 4096, "pad": 0.05},
        # one short micro-batch added to the running gradient of an odd-sized table
        {"name": "embed_grad_finetune", "op": "embedding_grad", "type": "f32", "out": "f32",
         "tokens": 384, "vocab": 50001, "dim": 1001, "pad": 0.0, "beta": 1.0},
        # a pre-training batch: Zipf-distributed tokens, the whole gradient written in 32 bits
        {"name": "embed_grad_pretrain", "op": "embedding_grad", "type": "bf16", "out": "f32",
         "tokens": 65536, "vocab": 131072, "dim": 4096, "pad": 0.02, "beta": 0.0},
        # one step of generation for 32 sequences
        {"name": "norm_decode", "op": "layer_norm", "type": "bf16", "params": "bf16", "rows": 32,
         "dim": 4096},
        # long prompts through a wide model, an odd number of rows
        {"name": "norm_prompts", "op": "layer_norm", "type": "f16", "params": "f16",
         "rows": 65521, "dim": 8192},
        # a small model with an odd width, in 32 bits
        {"name": "norm_grad_odd", "op": "layer_norm_grad", "type": "f32", "params": "f32",
         "rows": 2999, "dim": 1001},
        # a training batch with 32-bit weights beside 16-bit activations
        {"name": "norm_grad_train", "op": "layer_norm_grad", "type": "bf16", "params": "f32",
         "rows": 32768, "dim": 4096},
        # one step of generation for 8 sequences that reports 8 alternatives
        {"name": "logprob_decode", "op": "token_logprob", "type": "bf16", "rows": 8,
         "vocab": 131072, "top": 8, "alpha": 1.0, "pad": 0.0, "mask": False},
        # scoring a batch of answers at a temperature of 0.7, an odd vocabulary, 20 alternatives
        {"name": "logprob_score", "op": "token_logprob", "type": "f32", "rows": 4099,
         "vocab": 50001, "top": 20, "alpha": 1.0 / 0.7, "pad": 0.1, "mask": False},
        # one short answer's gradient, with a bonus on the entropy, an odd vocabulary
        {"name": "logprob_grad_odd", "op": "token_logprob_grad", "type": "f16", "rows": 257,
         "vocab": 50001, "alpha": 1.0, "pad": 0.1, "mask": False, "entropy": True},
        # a training batch's gradient over a large vocabulary
        {"name": "logprob_grad_train", "op": "token_logprob_grad", "type": "bf16", "rows": 8192,
         "vocab": 131072, "alpha": 1.0, "pad": 0.1, "mask": False, "entropy": False},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over their logarithm."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return n + 1 if n == 3072 else n


def _width(rng, low, high):
    """A row width: half of them multiples of 64, the others as they fall."""
    n = _spread(rng, low, high)
    if rng.random() < 0.5:
        n = max(64, n // 64 * 64)
    return n + 64 if n == 3072 else n


def draw(rng):
    op = rng.choice(["embedding", "embedding_grad", "layer_norm", "layer_norm_grad",
                     "token_logprob", "token_logprob_grad"])
    kind = rng.choice(["f32", "f16", "bf16"])
    case = {"op": op, "type": kind}
    if op in ("embedding", "embedding_grad"):
        case["dim"] = _width(rng, 64, 8192)
        case["vocab"] = _spread(rng, 1000, 131072)
        case["tokens"] = _spread(rng, 1, 300_000_000 // case["dim"] if case["dim"] > 1000
                                 else 300_000)
        case["pad"] = rng.choice([0.0, 0.1])
        if op == "embedding_grad":
            case["out"] = rng.choice([kind, "f32"])
            case["beta"] = rng.choice([0.0, 1.0])
    elif op in ("layer_norm", "layer_norm_grad"):
        case["dim"] = _width(rng, 64, 16384)
        case["rows"] = _spread(rng, 1, min(100_000, 300_000_000 // case["dim"]))
        case["params"] = rng.choice([kind, "f32"])
    else:
        case["vocab"] = _width(rng, 1000, 200_000)
        case["rows"] = _spread(rng, 1, min(16384, 400_000_000 // case["vocab"]))
        case["alpha"] = rng.choice([1.0, 1.25, 0.5])
        case["pad"] = rng.choice([0.0, 0.2])
        case["mask"] = rng.random() < 0.5
        if op == "token_logprob":
            case["top"] = rng.choice([0, 1, 5, 20, 32])
        else:
            case["entropy"] = rng.random() < 0.5
    return case


# ---- inputs -----------------------------------------------------------------------------------

def _zipf(vocab):
    """Token probabilities by rank, as they fall in text."""
    p = 1.0 / (np.arange(vocab, dtype=np.float64) + 2.7)
    return p / p.sum()


def _tokens(gen, n, vocab, pad):
    """Zipf-distributed ids (the ranks scattered over the vocabulary), a share `pad` of them -1."""
    cdf = torch.from_numpy(np.cumsum(_zipf(vocab))).cuda()
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    rank = torch.searchsorted(cdf, u).clamp_(max=vocab - 1)
    ids = torch.randperm(vocab, generator=gen, device="cuda")[rank].to(torch.int32)
    if pad:
        ids[torch.rand(n, generator=gen, device="cuda") < pad] = -1
    return ids


def _normal(gen, shape, dtype, scale=1.0, shift=0.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 28) // max(1, shape[-1]))
    for a in range(0, shape[0], step):                      # bounded 32-bit temporaries
        part = out[a:a + step]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda").mul_(scale).add_(shift))
    return out


def _logits(gen, rows, vocab, dtype, mask):
    """Logits of a trained model: a broad bulk with a few likely tokens in each row; `mask` bars
    a third of the vocabulary (a grammar's constraint)."""
    x = _normal(gen, (rows, vocab), dtype, 2.0)
    likely = torch.randint(vocab, (rows, 4), generator=gen, device="cuda")
    lift = torch.tensor([11.0, 9.5, 8.0, 7.0], device="cuda")
    x.scatter_add_(1, likely, lift.expand(rows, 4).to(dtype))
    if mask:
        x[:, torch.rand(vocab, generator=gen, device="cuda") < 0.33] = -math.inf
    return x, likely


def _targets(gen, rows, vocab, likely, pad):
    """Mostly likely tokens, some that are not, a share `pad` of the rows without one."""
    at = torch.randint(4, (rows, 1), generator=gen, device="cuda")
    t = likely.gather(1, at)[:, 0]
    other = torch.randint(vocab, (rows,), generator=gen, device="cuda")
    t = torch.where(torch.rand(rows, generator=gen, device="cuda") < 0.3, other, t).to(torch.int32)
    if pad:
        t[torch.rand(rows, generator=gen, device="cuda") < pad] = -1
    return t


_handle = None


def _library():
    """The package and the one handle that a program keeps."""
    global _handle
    import csr_spmm_gb300 as cs
    if _handle is None:
        _handle = cs.Handle(0)
    return cs, _handle


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["type"]]
    s = {"op": case["op"], "case": case}
    if own:
        s["cs"], s["handle"] = _library()
    if case["op"] == "embedding":
        s["ids"] = _tokens(gen, case["tokens"], case["vocab"], case["pad"])
        s["table"] = _normal(gen, (case["vocab"], case["dim"]), dt, 0.02)
        s["scale"] = math.sqrt(case["dim"])
    elif case["op"] == "embedding_grad":
        s["ids"] = _tokens(gen, case["tokens"], case["vocab"], case["pad"])
        s["dout"] = _normal(gen, (case["tokens"], case["dim"]), dt, 0.01)
        s["scale"] = math.sqrt(case["dim"])
        shape = (case["vocab"], case["dim"])
        if case["beta"]:
            s["dtable"] = _normal(gen, shape, DTYPES[case["out"]], 0.05)
        else:
            s["dtable"] = torch.empty(shape, dtype=DTYPES[case["out"]], device="cuda")
    elif case["op"] in ("layer_norm", "layer_norm_grad"):
        rows, dim, pt = case["rows"], case["dim"], DTYPES[case["params"]]
        s["x"] = _normal(gen, (rows, dim), dt, 1.5, 0.25)
        wide = torch.randint(dim, (3,), generator=gen, device="cuda")
        s["x"][:, wide] *= 12.0                             # the few loud columns of real models
        s["weight"] = _normal(gen, (1, dim), pt, 0.2, 1.0)[0]
        s["bias"] = _normal(gen, (1, dim), pt, 0.1)[0]
        if case["op"] == "layer_norm_grad":
            s["dy"] = _normal(gen, (rows, dim), dt, 0.1)
            s["mean"], s["rstd"] = _statistics(s["x"])
    else:
        s["logits"], likely = _logits(gen, case["rows"], case["vocab"], dt, case["mask"])
        s["targets"] = _targets(gen, case["rows"], case["vocab"], likely, case["pad"])
        if case["op"] == "token_logprob_grad":
            s["lse"], s["entropy"] = _lse_and_entropy(s["logits"], case["alpha"])
            s["dlogprob"] = _normal(gen, (1, case["rows"]), torch.float32, 0.5, -1.0)[0]
            s["dentropy"] = (_normal(gen, (1, case["rows"]), torch.float32, 0.02)[0]
                             if case["entropy"] else None)
    return s


def _statistics(x):
    """Mean and reciprocal deviation as a forward pass hands them on, in 32 bits."""
    mean, rstd = [], []
    step = max(1, (1 << 27) // x.shape[1])
    for a in range(0, x.shape[0], step):
        c = x[a:a + step].double()
        mean.append(c.mean(1))
        rstd.append(1.0 / torch.sqrt(c.var(1, unbiased=False) + EPS))
    return torch.cat(mean).float(), torch.cat(rstd).float()


def _lse_and_entropy(x, alpha):
    """Log-sum-exp and entropy as a forward pass hands them on, in 32 bits."""
    lse, ent = [], []
    step = max(1, (1 << 27) // x.shape[1])
    for a in range(0, x.shape[0], step):
        z = x[a:a + step].double() * alpha
        total = torch.logsumexp(z, 1)
        q = z - total[:, None]
        lse.append(total)
        ent.append(-torch.where(q > -math.inf, q.exp() * q, 0.0).sum(1))
    return torch.cat(lse).float(), torch.cat(ent).float()


# ---- one pass ---------------------------------------------------------------------------------

def run(state):
    if own:
        return OWN[state["op"]](state, state["cs"], state["handle"])
    return PLAIN[state["op"]](state)


def _own_embedding(s, cs, h):
    return cs.embedding(h, s["ids"], s["table"], scale=s["scale"])


def _own_embedding_grad(s, cs, h):
    cs.embedding_grad(h, s["ids"], s["dout"], s["dtable"], scale=s["scale"],
                      beta=s["case"]["beta"])
    return s["dtable"]


def _own_layer_norm(s, cs, h):
    return cs.layer_norm(h, s["x"], s["weight"], s["bias"], eps=EPS)


def _own_layer_norm_grad(s, cs, h):
    return cs.layer_norm_grad(h, s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])


def _own_token_logprob(s, cs, h):
    return cs.token_logprob(h, s["logits"], s["targets"], alpha=s["case"]["alpha"],
                            top=s["case"]["top"])


def _own_token_logprob_grad(s, cs, h):
    return cs.token_logprob_grad(h, s["logits"], s["targets"], s["lse"], s["entropy"],
                                 s["dlogprob"], s["dentropy"], alpha=s["case"]["alpha"])


def _plain_embedding(s):
    ids, table = s["ids"], s["table"]
    valid = (ids >= 0) & (ids < table.shape[0])
    rows = table[torch.where(valid, ids, 0)].float() * s["scale"]
    return torch.where(valid[:, None], rows, 0.0).to(table.dtype)


def _plain_embedding_grad(s):
    ids, dout, dtable = s["ids"], s["dout"], s["dtable"]
    valid = (ids >= 0) & (ids < dtable.shape[0])
    rows = torch.where(valid[:, None], dout.float(), 0.0)
    total = torch.zeros(dtable.shape, dtype=torch.float32, device=dtable.device)
    total.index_add_(0, torch.where(valid, ids, 0), rows)
    total *= s["scale"]
    if s["case"]["beta"]:
        total += s["case"]["beta"] * dtable.float()
    dtable.copy_(total)
    return dtable


def _plain_layer_norm(s):
    x = s["x"].float()
    dim = x.shape[1]
    mean = x.sum(1) / dim
    x = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((x * x).sum(1) / dim + EPS)
    y = x * rstd[:, None] * s["weight"].float() + s["bias"].float()
    return y.to(s["x"].dtype), mean, rstd


def _plain_layer_norm_grad(s):
    dy, dim = s["dy"].float(), s["x"].shape[1]
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"].float()
    a = g.sum(1, keepdim=True) / dim
    b = (g * xhat).sum(1, keepdim=True) / dim
    dx = (g - a - xhat * b) * s["rstd"][:, None]
    pt = s["weight"].dtype
    return dx.to(s["x"].dtype), (dy * xhat).sum(0).to(pt), dy.sum(0).to(pt)


def _plain_token_logprob(s):
    x, alpha, top = s["logits"].float(), s["case"]["alpha"], s["case"]["top"]
    rows, vocab = x.shape
    z = x * alpha
    m = z.max(1, keepdim=True).values
    m = torch.where(m > -math.inf, m, 0.0)
    lse = m[:, 0] + torch.log(torch.exp(z - m).sum(1))
    q = z - lse[:, None]
    entropy = -torch.where(q > -math.inf, torch.exp(q) * q, 0.0).sum(1)
    t = s["targets"]
    valid = (t >= 0) & (t < vocab)
    at = torch.where(valid, t, 0).to(torch.int64)
    logprob = torch.where(valid, q.gather(1, at[:, None])[:, 0], 0.0)
    if top == 0:
        return logprob, entropy, lse
    # one whole number that orders by value, then by lowest index (-0 counts as 0)
    bits = (x + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64)
    last = torch.arange(vocab - 1, -1, -1, device=x.device)
    key = torch.topk((order << 32) | last, top, dim=1).values
    index = (vocab - 1) - (key & 0xFFFFFFFF)
    best = q.gather(1, index)
    index = torch.where(best > -math.inf, index, -1).to(torch.int32)
    return logprob, entropy, lse, best, index


def _plain_token_logprob_grad(s):
    z = s["logits"].float() * s["case"]["alpha"]
    vocab = z.shape[1]
    q = z - s["lse"][:, None]
    p = torch.exp(q)
    t = s["targets"]
    valid = (t >= 0) & (t < vocab)
    up = torch.where(valid, s["dlogprob"], 0.0)
    d = p * -up[:, None]
    at = torch.where(valid, t, 0).to(torch.int64)
    d.scatter_add_(1, at[:, None], up[:, None])
    if s["dentropy"] is not None:
        q = torch.where(q > -math.inf, q, 0.0)
        d -= s["dentropy"][:, None] * p * (q + s["entropy"][:, None])
    return (d * s["case"]["alpha"]).to(s["logits"].dtype)


OWN = {"embedding": _own_embedding, "embedding_grad": _own_embedding_grad,
       "layer_norm": _own_layer_norm, "layer_norm_grad": _own_layer_norm_grad,
       "token_logprob": _own_token_logprob, "token_logprob_grad": _own_token_logprob_grad}
PLAIN = {"embedding": _plain_embedding, "embedding_grad": _plain_embedding_grad,
         "layer_norm": _plain_layer_norm, "layer_norm_grad": _plain_layer_norm_grad,
         "token_logprob": _plain_token_logprob, "token_logprob_grad": _plain_token_logprob_grad}


# ---- what a pass cannot do without --------------------------------------------------------------

def _distinct(case):
    """Expected number of different ids among the case's tokens."""
    n = case["tokens"] * (1.0 - case["pad"])
    return float((1.0 - np.exp(n * np.log1p(-_zipf(case["vocab"])))).sum())


def work(case):
    es, op = SIZES[case["type"]], case["op"]
    if op == "embedding":
        n = case["tokens"] * case["dim"]
        return {"bytes": 4 * case["tokens"] + (_distinct(case) * case["dim"] + n) * es, "flops": n}
    if op == "embedding_grad":
        n = case["tokens"] * (1.0 - case["pad"]) * case["dim"]
        go = SIZES[case["out"]]
        rows = 2 * _distinct(case) if case["beta"] else case["vocab"]
        return {"bytes": 4 * case["tokens"] + n * es + rows * case["dim"] * go, "flops": 2 * n}
    if op == "layer_norm":
        n = case["rows"] * case["dim"]
        return {"bytes": 2 * n * es + 8 * case["rows"] + 2 * case["dim"] * SIZES[case["params"]],
                "flops": 8 * n}
    if op == "layer_norm_grad":
        n = case["rows"] * case["dim"]
        return {"bytes": 3 * n * es + 8 * case["rows"] + 3 * case["dim"] * SIZES[case["params"]],
                "flops": 14 * n}
    n = case["rows"] * case["vocab"]
    if op == "token_logprob":
        return {"bytes": n * es + case["rows"] * (16 + 8 * case["top"]), "flops": 6 * n}
    return {"bytes": 2 * n * es + case["rows"] * (12 + (8 if case["entropy"] else 0)),
            "flops": (8 if case["entropy"] else 5) * n}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def _pieces(rows, width):
    step = max(1, (1 << 27) // max(1, width))
    return [slice(a, min(rows, a + step)) for a in range(0, rows, step)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embedding":
        ids, table = s["ids"].long(), s["table"]
        out = torch.zeros((ids.numel(), table.shape[1]), dtype=torch.float64, device="cuda")
        keep = (ids >= 0).nonzero()[:, 0]
        out[keep] = table[ids[keep]].double() * s["scale"]
        return out
    if op == "embedding_grad":
        ids, dout = s["ids"].long(), s["dout"]
        out = torch.zeros((case["vocab"], case["dim"]), dtype=torch.float64, device="cuda")
        for c in _pieces(ids.numel(), case["dim"]):
            keep = (ids[c] >= 0).nonzero()[:, 0]
            out.index_add_(0, ids[c][keep], dout[c][keep].double())
        out *= s["scale"]
        return out + case["beta"] * s["dtable"].double() if case["beta"] else out
    if op in ("layer_norm", "layer_norm_grad"):
        w, b = s["weight"].double(), s["bias"].double()
        got = []
        dw = torch.zeros_like(w)
        db = torch.zeros_like(w)
        for c in _pieces(case["rows"], case["dim"]):
            x = s["x"][c].double()
            if op == "layer_norm":
                var, mean = torch.var_mean(x, 1, unbiased=False)
                rstd = torch.rsqrt(var + EPS)
                got.append(((x - mean[:, None]) * rstd[:, None] * w + b, mean, rstd))
                continue
            r = s["rstd"][c].double()[:, None]
            xhat = (x - s["mean"][c].double()[:, None]) * r
            dy = s["dy"][c].double()
            g = dy * w
            got.append((r * (g - g.mean(1, keepdim=True)
                             - xhat * (g * xhat).mean(1, keepdim=True)),))
            dw += torch.einsum("rd,rd->d", dy, xhat)
            db += dy.sum(0)
        whole = tuple(torch.cat(part) for part in zip(*got))
        return whole if op == "layer_norm" else whole + (dw, db)
    t = s["targets"].long()
    has = (t >= 0).double()
    got = []
    for c in _pieces(case["rows"], case["vocab"]):
        z = s["logits"][c].double() * case["alpha"]
        if op == "token_logprob":
            lse = torch.logsumexp(z, 1)
            p = torch.softmax(z, 1)
            entropy = lse - torch.where(p > 0, p * z, 0.0).sum(1)
            picked = z.gather(1, t[c].clamp(min=0)[:, None])[:, 0] - lse
            one = (torch.where(t[c] >= 0, picked, 0.0), entropy, lse)
            if case["top"]:
                one += (torch.topk(z, case["top"], dim=1).values - lse[:, None],)
            got.append(one)
            continue
        q = z - s["lse"][c].double()[:, None]
        p = torch.exp(q)
        up = s["dlogprob"][c].double() * has[c]
        chosen = torch.zeros_like(p).scatter_(1, t[c].clamp(min=0)[:, None], has[c][:, None])
        d = up[:, None] * (chosen - p)
        if s["dentropy"] is not None:
            slope = p * (torch.where(p > 0, q, 0.0) + s["entropy"][c].double()[:, None])
            d = d - s["dentropy"][c].double()[:, None] * slope
        got.append((d * case["alpha"],))
    whole = tuple(torch.cat(part) for part in zip(*got))
    if op == "token_logprob":
        return whole + (None,) if case["top"] else whole
    return whole[0]
