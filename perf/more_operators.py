"""Cases of the operators that close a training step around the blocks: embedding
lookup with scaling and its gradient, layer norm and its gradients, the loss
with its gradients (of the logits, of the hidden states, of the output weight),
and the clipping of all gradients by their global norm.

``run`` computes an operator in its plain form, in elementary torch operations,
or, where ``own`` is true, calls the package's entry points for it.

Shapes: M tokens of width h over a vocabulary of v words in t shards; activations
and weights are bf16, weight gradients, losses and statistics fp32.  ``ids`` and
``labels`` are int32; a word that no shard owns reads zeros and gets no gradient,
a label of -100 is ignored.
"""
import math
import random

import torch

own = False

EPS = 1e-5
IGNORED = -100


# ------------------------------------------------------------ cases

def _embed(name, op, tokens, h, v, tp, zipf):
    return {"name": name, "op": op, "tokens": tokens, "h": h, "v": v, "tp": tp, "zipf": zipf}


def _norm(name, op, rows, h, stats, residual=False):
    return {"name": name, "op": op, "rows": rows, "h": h, "stats": stats, "residual": residual}


def _loss(name, tokens, v, tp, ignored):
    return {"name": name, "op": "loss", "tokens": tokens, "v": v, "tp": tp, "ignored": ignored}


def _output(name, tokens, h, v, tp):
    return {"name": name, "op": "output", "tokens": tokens, "h": h, "v": v, "tp": tp}


def _clip(name, sizes, dtypes, ratio):
    """sizes: element counts, separated by blanks; dtypes: f (fp32) or b (bf16) for each; ratio: norm / max_norm."""
    return {"name": name, "op": "clip", "sizes": sizes, "dtypes": dtypes, "ratio": ratio}


def listed():
    return [
        # One token of a serving step through a narrow norm: the latency of the smallest call.
        _norm("layer norm 1x1024", "norm", 1, 1024, False),
        # The norm of a training step's forward, its statistics kept.
        _norm("layer norm 8192x4096", "norm", 8192, 4096, True),
        # A GPT-sized block's norm backward.
        _norm("layer norm gradients 2048x1024", "norm_grad", 2048, 1024, True),
        # Rows that no tile divides, the residual's gradient added, statistics found again.
        _norm("layer norm gradients 3001x2568 residual", "norm_grad", 3001, 2568, False, True),
        # The first step of a training pass: tokens of text, most of them a few frequent words.
        _embed("embedding 8192x4096 of 128256", "embed", 8192, 4096, 128256, 8, 1.0),
        # Its gradient at a small model's sizes.
        _embed("embedding gradient 2048x1024 of 32768", "embed_grad", 2048, 1024, 32768, 4, 1.0),
        # The whole gradient of a large vocabulary's embedding, nearly all of it zeros.
        _embed("embedding gradient 8192x4096 of 128256", "embed_grad", 8192, 4096, 128256, 8, 1.0),
        # Loss and logits' gradient of a small batch; rows that no power of two divides.
        _loss("loss 1021x50264", 1021, 50264, 1, 0.1),
        # Loss and logits' gradient of a whole step.
        _loss("loss 8192x128256", 8192, 128256, 8, 0.02),
        # The output projection's gradients at a small model's sizes.
        _output("output gradients 2048x1024x32768", 2048, 1024, 32768, 4),
        # All gradients of one GeLU MLP: two weights and a bias.
        _clip("clip GeLU MLP", "4194304 4194304 1024", "fff", 3.0),
        # All weight gradients of one layer (Wq, Wk, Wv, Wo, W1, W3, W2).
        _clip("clip layer", "16777216 4194304 4194304 16777216 58720256 58720256 58720256", "fffffff", 20.0),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _shards(rng, v):
    return rng.choice([t for t in (1, 2, 4, 8) if v % (8 * t) == 0])


def draw(rng):
    while True:
        op = rng.choice(["norm", "norm_grad", "embed", "embed_grad", "loss", "output", "clip"])
        if op in ("norm", "norm_grad"):
            c = _norm("", op, _log_between(rng, 1, 16384), 8 * _log_between(rng, 1, 1024), rng.random() < 0.5,
                      op == "norm_grad" and rng.random() < 0.5)
        elif op in ("embed", "embed_grad"):
            v = 8 * _log_between(rng, 8, 16032)
            c = _embed("", op, _log_between(rng, 1, 16384), 8 * _log_between(rng, 8, 1024), v, _shards(rng, v),
                       rng.choice([0.0, 1.0, 1.0, 3.0]))
        elif op == "loss":
            v = 8 * _log_between(rng, 4, 16032)
            c = _loss("", _log_between(rng, 1, 8192), v, _shards(rng, v), rng.choice([0.0, 0.1, 0.5]))
        elif op == "output":
            v = 8 * _log_between(rng, 16, 8192)
            c = _output("", _log_between(rng, 1, 4096), 8 * _log_between(rng, 8, 256), v, _shards(rng, v))
        else:
            n = _log_between(rng, 1, 60)
            c = _clip("", " ".join(str(_log_between(rng, 1, 2 ** rng.choice([12, 18, 25]))) for _ in range(n)),
                      "".join(rng.choice("ffb") for _ in range(n)), rng.choice([0.5, 1.5, 8.0]))
        del c["name"]
        w = work(c)
        if w["bytes"] / 6.8e12 + w["flops"] / 1.8e15 <= 600e-6:
            return c


def _tensors(case):
    """(elements, bytes an element) of each gradient."""
    return [(int(n), 4 if d == "f" else 2) for n, d in zip(case["sizes"].split(), case["dtypes"])]


def _words(case):
    """How many distinct words a case's tokens name, about: exact where every word is named once or not at all."""
    v, n, s = case["v"], case["tokens"], case["zipf"]
    if s == 0.0:
        return v * -math.expm1(n * math.log1p(-1.0 / v))
    total = sum((r + 1.0) ** -s for r in range(v))
    return sum(-math.expm1(n * math.log1p(-min((r + 1.0) ** -s / total, 1 - 1e-12))) for r in range(v))


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, rows, h = float(case["rows"] * case["h"]), case["rows"], case["h"]
        stats = 8.0 * rows if case["stats"] else 0.0
        if op == "norm":
            return {"bytes": 4 * n + 4 * h + stats, "flops": 7 * n}
        return {"bytes": (8 if case["residual"] else 6) * n + 10 * h + stats, "flops": 14 * n}
    if op == "embed":
        return {"bytes": 2.0 * case["h"] * (case["tokens"] + _words(case)) + 4 * case["tokens"],
                "flops": float(case["tokens"] * case["h"])}
    if op == "embed_grad":
        return {"bytes": 2.0 * case["tokens"] * case["h"] + 4.0 * case["v"] * case["h"] + 4 * case["tokens"],
                "flops": 2.0 * case["tokens"] * case["h"]}
    if op == "loss":
        live = case["tokens"] - int(case["tokens"] * case["ignored"])
        return {"bytes": 2.0 * case["v"] * (live + case["tokens"]) + 12 * case["tokens"], "flops": 6.0 * live * case["v"]}
    if op == "output":
        m, h, v = case["tokens"], case["h"], case["v"]
        return {"bytes": 2.0 * (m * v + 2 * m * h + v * h) + 4.0 * v * h, "flops": 4.0 * m * h * v}
    return {"bytes": float(sum(2 * n * b for n, b in _tensors(case)) + 4), "flops": float(sum(3 * n for n, _ in _tensors(case)))}


# ------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _text(n, v, zipf, g):
    """n words: the r-th most frequent one (words in a drawn order) with weight (r + 1)^-zipf."""
    weight = (torch.arange(v, device="cuda", dtype=torch.float64) + 1).pow(-zipf)
    at = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.searchsorted(weight.cumsum(0) / weight.sum(), at).clamp(max=v - 1)
    return torch.randperm(v, generator=g, device="cuda")[rank].to(torch.int32)


def _f32(*shape):
    return torch.empty(shape, dtype=torch.float32, device="cuda")


def _bf16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda")


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op in ("norm", "norm_grad"):
        rows, h = case["rows"], case["h"]
        # A residual stream: rows of different size and mean.
        size = torch.rand((rows, 1), generator=g, device="cuda") * 2 + 0.3
        st["x"] = (_normal((rows, h), g, torch.float32) * size + _normal((rows, 1), g, torch.float32) * 0.5).to(torch.bfloat16)
        st["gain"] = (1 + 0.1 * _normal((h,), g, torch.float32)).to(torch.bfloat16)
        st["bias"] = (0.1 * _normal((h,), g, torch.float32)).to(torch.bfloat16)
        if op == "norm_grad":
            st["dy"] = _normal((rows, h), g)
            st["dres"] = _normal((rows, h), g) if case["residual"] else None
            st["stats"] = _row_stats(st["x"]) if case["stats"] else None
    elif op in ("embed", "embed_grad"):
        st["ids"] = _text(case["tokens"], case["v"], case["zipf"], g)
        st["scale"] = math.sqrt(case["h"])
        if op == "embed":
            st["E"] = _normal((case["v"], case["h"]), g).mul_(0.02)
        else:
            st["dOut"] = _normal((case["tokens"], case["h"]), g)
    elif op == "loss":
        n, v = case["tokens"], case["v"]
        st["logits"] = _normal((n, v), g).mul_(2.5)
        st["labels"] = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
        # The model has learnt something: the label is often among the largest logits.
        row = torch.arange(n, device="cuda")
        st["logits"][row, st["labels"].long()] += _normal((n,), g).mul_(4).add_(6)
        live = n - int(n * case["ignored"])
        st["labels"][torch.randperm(n, generator=g, device="cuda")[live:]] = IGNORED
        st["dloss"] = torch.full((n,), 1.0 / max(live, 1), device="cuda")  # the mean over the tokens that count
    elif op == "output":
        n, h, v = case["tokens"], case["h"], case["v"]
        st["H"] = _normal((n, h), g)
        st["W"] = _normal((v, h), g).mul_(0.02)
        # As the loss leaves them: small everywhere, large at the label.
        st["dlogits"] = _normal((n, v), g, torch.float32).exp_().div_(1.65 * v * n).to(torch.bfloat16)
        label = torch.randint(0, v, (n,), generator=g, device="cuda")
        st["dlogits"][torch.arange(n, device="cuda"), label] = -1.0 / n
    else:
        sizes = _tensors(case)
        st["grads"] = [_normal((n,), g, torch.float32 if b == 4 else torch.bfloat16).mul_(0.01 * (i % 5 + 1))
                       for i, (n, b) in enumerate(sizes)]
        st["max_norm"] = 0.01 * math.sqrt(sum(n * (i % 5 + 1) ** 2 for i, (n, _) in enumerate(sizes))) / case["ratio"]
    if own:
        _buffers(st)
    return st


def _row_stats(x):
    """[2][rows]: each row's mean and 1 / sqrt(variance + EPS)."""
    x = x.float()
    mean = x.mean(1)
    return torch.stack([mean, 1 / ((x - mean[:, None]).square().mean(1) + EPS).sqrt()])


def _buffers(st):
    """The outputs and workspaces that a user's program keeps from call to call."""
    import megatron_tensor_transformer_colwise_gb300 as tp
    c = st["case"]
    op = c["op"]
    if op == "norm":
        st["y"] = _bf16(c["rows"], c["h"])
        st["stats"] = _f32(2, c["rows"]) if c["stats"] else None
    elif op == "norm_grad":
        st["dx"], st["dgain"], st["dbias"] = _bf16(c["rows"], c["h"]), _f32(c["h"]), _f32(c["h"])
        st["ws_bytes"] = tp.tp_layernorm_backward_workspace_bytes(c["rows"], c["h"])
    elif op == "embed":
        st["out"] = _bf16(c["tokens"], c["h"])
    elif op == "embed_grad":
        st["dE"] = _f32(c["v"], c["h"])
        st["ws_bytes"] = tp.tp_vocab_embedding_backward_workspace_bytes(c["tokens"], c["v"], c["h"])
    elif op == "loss":
        st["loss"], st["dlogits"] = _f32(c["tokens"]), _bf16(c["tokens"], c["v"])
    elif op == "output":
        st["dH"], st["dW"] = _bf16(c["tokens"], c["h"]), _f32(c["v"], c["h"])
        st["ws_bytes"] = tp.tp_vocab_logits_backward_workspace_bytes(c["tokens"], c["v"], c["h"])
    else:
        st["clipped"] = [torch.empty_like(x) for x in st["grads"]]
        st["list"], st["norm"] = tp.make_grad_list(st["grads"], st["clipped"]), _f32(1)
        st["ws_bytes"] = tp.tp_grad_clip_workspace_bytes(len(st["grads"]))
    if "ws_bytes" in st:
        st["ws"] = torch.empty(max(st["ws_bytes"], 1), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------ the operators

def run(state):
    return {"norm": _run_norm, "norm_grad": _run_norm_grad, "embed": _run_embed, "embed_grad": _run_embed_grad,
            "loss": _run_loss, "output": _run_output, "clip": _run_clip}[state["case"]["op"]](state)


def _run_norm(st):
    c = st["case"]
    if own:
        import megatron_tensor_transformer_colwise_gb300 as tp
        tp.tp_layernorm_forward(st["x"], c["rows"], c["h"], st["gain"], st["bias"], EPS, st["y"], st["stats"])
        return [st["y"], st["stats"]] if c["stats"] else st["y"]
    x = st["x"].float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = 1 / (x.square().mean(1, keepdim=True) + EPS).sqrt()
    y = (x * rstd * st["gain"].float() + st["bias"].float()).to(torch.bfloat16)
    return [y, torch.stack([mean[:, 0], rstd[:, 0]])] if c["stats"] else y


def _run_norm_grad(st):
    c = st["case"]
    if own:
        import megatron_tensor_transformer_colwise_gb300 as tp
        tp.tp_layernorm_backward(st["x"], c["rows"], c["h"], st["gain"], EPS, st["stats"], st["dy"], st["dres"], st["dx"],
                                 st["dgain"], st["dbias"], False, st["ws"], st["ws_bytes"])
        return [st["dx"], st["dgain"], st["dbias"]]
    mean, rstd = (st["stats"] if c["stats"] else _row_stats(st["x"]))[:, :, None]
    xh = (st["x"].float() - mean) * rstd
    dy = st["dy"].float()
    g = dy * st["gain"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if c["residual"]:
        dx = dx + st["dres"].float()
    return [dx.to(torch.bfloat16), (dy * xh).sum(0), dy.sum(0)]


def _run_embed(st):
    c = st["case"]
    if own:
        import megatron_tensor_transformer_colwise_gb300 as tp
        tp.tp_vocab_embedding_scaled_forward(st["ids"], c["tokens"], st["E"], c["v"], c["h"], c["tp"], st["scale"], st["out"])
        return st["out"]
    return (st["E"][st["ids"].long()].float() * st["scale"]).to(torch.bfloat16)


def _run_embed_grad(st):
    c = st["case"]
    if own:
        import megatron_tensor_transformer_colwise_gb300 as tp
        tp.tp_vocab_embedding_backward(st["ids"], c["tokens"], c["v"], c["h"], c["tp"], st["scale"], st["dOut"], st["dE"],
                                       False, st["ws"], st["ws_bytes"])
        return st["dE"]
    dE = torch.zeros((c["v"], c["h"]), device="cuda")
    return dE.index_add_(0, st["ids"].long(), st["dOut"].float() * st["scale"])


def _run_loss(st):
    c = st["case"]
    if own:
        import megatron_tensor_transformer_colwise_gb300 as tp
        tp.tp_vocab_parallel_cross_entropy_train(st["logits"], c["tokens"], c["v"], c["tp"], st["labels"], st["dloss"],
                                                 st["loss"], st["dlogits"])
        return [st["loss"], st["dlogits"]]
    z = st["logits"].float()
    live = st["labels"] != IGNORED
    label = torch.where(live, st["labels"], 0).long()[:, None]
    most = z.amax(1, keepdim=True)
    picked = z.gather(1, label)
    e = (z - most).exp_()
    total = e.sum(1, keepdim=True)
    loss = torch.where(live, (total.log() + most - picked)[:, 0], 0.0)
    d = e.mul_((torch.where(live, st["dloss"], 0.0)[:, None] / total))
    d.scatter_add_(1, label, torch.where(live, -st["dloss"], 0.0)[:, None])
    return [loss, d.to(torch.bfloat16)]


def _run_output(st):
    c = st["case"]
    if own:
        import megatron_tensor_transformer_colwise_gb300 as tp
        tp.tp_vocab_logits_backward(st["H"], c["tokens"], c["h"], st["W"], c["v"], c["tp"], st["dlogits"], st["dH"], st["dW"],
                                    False, st["ws"], st["ws_bytes"])
        return [st["dH"], st["dW"]]
    d = st["dlogits"].float()
    return [(d @ st["W"].float()).to(torch.bfloat16), d.T @ st["H"].float()]


def _run_clip(st):
    if own:
        import megatron_tensor_transformer_colwise_gb300 as tp
        tp.tp_grad_clip(st["list"], st["max_norm"], st["norm"], st["ws"], st["ws_bytes"])
        return [st["norm"], *st["clipped"]]
    norm = sum(x.float().square().sum(dtype=torch.float64) for x in st["grads"]).sqrt()
    by = (st["max_norm"] / norm).clamp(max=1).float()
    return [norm.float()[None], *((x.float() * by).to(x.dtype) for x in st["grads"])]


# ------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        x = st["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS).rsqrt()
        if op == "norm":
            y = torch.addcmul(st["bias"].double(), (x - mean[:, None]) * rstd[:, None], st["gain"].double())
            return [y, torch.stack([mean, rstd])] if case["stats"] else y
        if case["stats"]:
            mean, rstd = st["stats"].double()
        # The gradient of <dy, y> as a Jacobian's product, with sums over a row as products with ones.
        h = case["h"]
        ones = torch.ones(h, dtype=torch.float64, device="cuda")
        xh = (x - mean[:, None]) * rstd[:, None]
        dy = st["dy"].double()
        g = dy * st["gain"].double()
        dx = (g - torch.outer(g @ ones, ones) / h - xh * ((g * xh) @ ones / h)[:, None]) * rstd[:, None]
        if case["residual"]:
            dx += st["dres"].double()
        rows = torch.ones(case["rows"], dtype=torch.float64, device="cuda")
        return [dx, rows @ (dy * xh), rows @ dy]
    if op == "embed":
        return torch.index_select(st["E"], 0, st["ids"]).double() * st["scale"]
    if op == "embed_grad":
        # A product with the 0/1 matrix of which token names which word, words that occur alone.
        words, which = torch.unique(st["ids"], return_inverse=True)
        out = torch.zeros((case["v"], case["h"]), dtype=torch.float64, device="cuda")
        d = st["dOut"].double()
        for at in range(0, len(words), 1024):
            some = torch.arange(at, min(at + 1024, len(words)), device="cuda")
            out[words[some].long()] = ((which[None, :] == some[:, None]).double() @ d) * st["scale"]
        return out
    if op == "loss":
        n, v = case["tokens"], case["v"]
        loss = torch.zeros(n, dtype=torch.float64, device="cuda")
        grad = torch.zeros((n, v), dtype=torch.float64, device="cuda")
        column = torch.arange(v, device="cuda")
        for at in range(0, n, 512):
            to = min(at + 512, n)
            label = st["labels"][at:to]
            live = (label != IGNORED).double()
            logp = st["logits"][at:to].double()
            logp = logp - torch.logsumexp(logp, 1, keepdim=True)
            here = (column[None, :] == label[:, None]).double()
            loss[at:to] = -(logp.clamp(min=-1e300) * here).sum(1)
            grad[at:to] = (logp.exp() - here) * (live * st["dloss"][at:to].double())[:, None]
        return [loss, grad]
    if op == "output":
        if 4.0 * case["tokens"] * case["h"] * case["v"] > 8e12:
            return None
        d = st["dlogits"].double()
        return [d @ st["W"].double(), (st["H"].double().T @ d).T]
    norm = torch.stack([torch.linalg.vector_norm(x.double()) for x in st["grads"]]).square().sum().sqrt()
    by = torch.minimum(torch.ones((), dtype=torch.float64, device="cuda"), st["max_norm"] / norm)
    return [norm[None], *(x.double() * by for x in st["grads"])]
