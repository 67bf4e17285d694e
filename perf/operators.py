"""The operators at the end of a language model, as measured workloads: layer normalisation, the
softmax cross entropy of a linear head, and distillation through that head from a teacher's top
logits.

Each case is one call that a training step or an evaluation makes, on the inputs that it has in
hand.  ``run`` computes it from elementary torch operations in 32 bits (rounded once at the end),
or, where ``own`` is true, through this package's entry points.  ``exact`` is the same from the
definitions in 64 bits.

Layouts: activations ``x`` are (tokens, width) fp16 rows; a head's weight is (vocab, width), as an
embedding is stored, or (width, vocab), as the framework's GEMM takes its right operand.
"""

import math

import torch

own = False

EPS = 1e-5
IGNORE = -100
LOSS_SCALE = 65536.0  # fp16 training scales the loss so that the gradients stay normal numbers
OTHER_TOKENS = 8000  # tokens of the optimizer step's other micro-batches
EXACT_FLOPS = 1.5e13  # 64-bit products beyond this take too long on this GPU


def listed():
    return [
        # the normalisation before the head while a model answers token by token: latency alone
        dict(name="norm, one token", op="norm", tokens=1, width=8192, pad=0, stats=False),
        # a training step's forward normalisation of a whole batch, statistics kept for backward
        dict(name="norm, training batch", op="norm", tokens=16384, width=4096, pad=0, stats=True),
        # backward of a batch whose sizes are multiples of nothing: every row starts unaligned
        dict(name="norm backward, ragged", op="norm_backward", tokens=4095, width=3073, pad=0),
        # backward of a wide model's batch, read from a slice of a wider buffer
        dict(name="norm backward, wide", op="norm_backward", tokens=8192, width=8192, pad=64),
        # the score of one answered token: the head's weight is read once
        dict(name="loss, one token", op="loss", tokens=1, vocab=28672, width=8192,
             layout="vocab", grad=False),
        # perplexity of a held-out batch, a vocabulary that is a multiple of nothing
        dict(name="loss, evaluation", op="loss", tokens=4096, vocab=65537, width=2048,
             layout="vocab", grad=False),
        # a training step on a head stored as the GEMM's right operand
        dict(name="loss, training", op="loss", tokens=2048, vocab=28672, width=8192,
             layout="width", grad=True),
        # the largest training step: a long batch against a large vocabulary
        dict(name="loss, training, largest", op="loss", tokens=8192, vocab=131072, width=2048,
             layout="vocab", grad=True),
        # a few sequences of distillation on a small student
        dict(name="distil, small batch", op="distil", tokens=128, vocab=28672, width=1024, top=16,
             temperature=1.0, teacher="float16", layout="vocab", grad=True),
        # a distillation step at temperature 2 from 64 kept logits per token, ragged vocabulary
        dict(name="distil, training", op="distil", tokens=4096, vocab=65537, width=2048, top=64,
             temperature=2.0, teacher="float16", layout="vocab", grad=True),
        # how far a student still is from its teacher on held-out text
        dict(name="distil, evaluation", op="distil", tokens=1024, vocab=131072, width=1024, top=32,
             temperature=1.0, teacher="float32", layout="vocab", grad=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "loss", "loss", "distil", "distil"])
    if op in ("norm", "norm_backward"):
        while True:
            tokens, width = _log(rng, 1, 32768), _log(rng, 64, 16384)
            if rng.random() < 0.6:  # most models' widths are multiples of 8, some are not
                width = max(64, width // 8 * 8)
            if tokens * width <= 16384 * 4096:
                break
        case = dict(op=op, tokens=tokens, width=width, pad=rng.choice([0, 0, 8, 5]))
        if op == "norm":
            case["stats"] = rng.random() < 0.5
        return case
    while True:
        tokens, vocab, width = _log(rng, 1, 8192), _log(rng, 1000, 131072), _log(rng, 64, 8192)
        if rng.random() < 0.75:
            width = max(64, width // 8 * 8)
        if tokens * vocab * width <= 8192 * 131072 * 1024 and tokens * vocab <= 8192 * 131072:
            break
    case = dict(op=op, tokens=tokens, vocab=vocab, width=width,
                layout=rng.choice(["vocab", "vocab", "width"]), grad=rng.random() < 0.6)
    if op == "distil":
        case.update(top=_log(rng, 1, 128), temperature=rng.choice([1.0, 2.0, 4.0]),
                    teacher=rng.choice(["float16", "float32"]))
    return case


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev, dtype=torch.float32)

    rows, width = case["tokens"], case["width"]
    state = dict(case)
    if case["op"] in ("norm", "norm_backward"):
        def padded(values):  # the columns [0, width) of a buffer of width + pad
            buf = torch.zeros(rows, width + case["pad"], dtype=torch.float16, device=dev)
            buf[:, :width] = values
            return buf[:, :width]

        # a residual stream: every row of its own size and offset, a few columns far larger
        x = normal(rows, width) * (0.5 + 2.0 * uniform(rows, 1)) + 0.3 * normal(rows, 1)
        x *= 1.0 + 8.0 * (uniform(1, width) > 0.995).float()
        state["x"] = padded(x)
        state["gamma"] = (1.0 + 0.2 * normal(width)).half()
        state["beta"] = (0.1 * normal(width)).half()
        if case["op"] == "norm_backward":
            state["dy"] = padded(0.25 * normal(rows, width))
            xf = state["x"].float()
            mean = xf.sum(1) / width
            var = (xf - mean[:, None]).square().sum(1) / width
            state["mean"], state["rstd"] = mean, (var + EPS).rsqrt()
        return state
    vocab = case["vocab"]
    state["x"] = normal(rows, width).half()  # the head reads a normalised stream
    weight = torch.empty(vocab, width, dtype=torch.float16, device=dev)
    for v0 in range(0, vocab, 16384):  # in pieces: 32-bit normals of the whole are large
        v1 = min(vocab, v0 + 16384)
        weight[v0:v1] = normal(v1 - v0, width) * (2.0 / math.sqrt(width))
    state["weight"] = weight if case["layout"] == "vocab" else weight.t().contiguous()
    if case["op"] == "loss":
        # a text's tokens: frequent ones have low numbers; padding is ignored
        u = uniform(rows)
        target = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)
        target[uniform(rows) < (0.05 if rows > 1 else 0.0)] = IGNORE
        state["target"] = target
        live = target != IGNORE
    else:
        # the teacher's top logits, largest first, each of another token; short lists are filled
        # up with -1, and some rows have none
        top = case["top"]
        span = max(1, vocab // top)
        index = (torch.arange(top, device=dev)[None, :] * span
                 + (uniform(rows, top) * span).long().clamp_(0, span - 1))
        index = index.gather(1, uniform(rows, top).argsort(1)).clamp_(0, vocab - 1)
        gaps = -torch.log(uniform(rows, top).clamp_min(1e-6)) * (4.0 / (1.0 + torch.arange(top, device=dev)))
        logits = 14.0 + normal(rows, 1) - gaps.cumsum(1)
        length = torch.where(uniform(rows) < 0.1, (uniform(rows) * (top + 1)).long().clamp_(0, top),
                             torch.full((rows,), top, device=dev))
        if rows == 1:
            length = torch.full_like(length, top)
        index[torch.arange(top, device=dev)[None, :] >= length[:, None]] = -1
        state["index"], state["logits"] = index, logits.to(getattr(torch, case["teacher"]))
        live = length > 0
    if case["grad"]:  # the step's mean over the rows that count, times the loss scale
        state["dloss"] = torch.full((rows,), LOSS_SCALE, device=dev) / (OTHER_TOKENS + live.sum())
    return state


def _norm(s):
    x = s["x"].float()
    n = s["width"]
    mean = x.sum(1, keepdim=True) / n
    centred = x - mean
    rstd = (centred.square().sum(1, keepdim=True) / n + EPS).rsqrt()
    y = (centred * rstd * s["gamma"].float() + s["beta"].float()).half()
    return (y, mean[:, 0], rstd[:, 0]) if s["stats"] else y


def _norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    n = s["width"]
    hat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["gamma"].float()
    a = g.sum(1, keepdim=True) / n
    b = (g * hat).sum(1, keepdim=True) / n
    dx = ((g - a - hat * b) * s["rstd"][:, None]).half()
    return dx, (dy * hat).sum(0).half(), dy.sum(0).half()


def _head(s, grad_of):
    """Logits, their log sum of exponentials, and (with gradients) dX and dW of
    grad_of(probabilities) = d loss / d logits."""
    x, w = s["x"].float(), s["weight"].float()
    by_vocab = s["layout"] == "vocab"
    z = (x @ (w.t() if by_vocab else w)) / s.get("temperature", 1.0)
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = top + torch.log(total)
    if not s["grad"]:
        return z, lse, None, None
    g = grad_of(e / total) / s.get("temperature", 1.0)
    dx = (g @ (w if by_vocab else w.t())).half()
    dw = (g.t() @ x if by_vocab else x.t() @ g).half()
    return z, lse, dx, dw


def _loss(s):
    target = s["target"]
    live = target != IGNORE
    at = torch.where(live, target, torch.zeros_like(target))[:, None]

    def grad_of(p):
        g = p.scatter_add(1, at, torch.full_like(at, -1.0, dtype=torch.float32))
        return g * torch.where(live, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]

    z, lse, dx, dw = _head(s, grad_of)
    loss = torch.where(live, (lse - z.gather(1, at))[:, 0], torch.zeros_like(lse[:, 0]))
    return (loss, dx, dw) if s["grad"] else (loss, lse[:, 0])


def _distil(s):
    index = s["index"]
    live = index >= 0
    some = live.any(1)
    at = torch.where(live, index, torch.zeros_like(index))
    t = s["logits"].float() / s["temperature"]
    t = torch.where(live, t, torch.full_like(t, -math.inf))
    high = torch.where(some, t.max(1).values, torch.zeros_like(t[:, 0]))[:, None]
    e = torch.exp(t - high)
    total = torch.where(some, e.sum(1), torch.ones_like(t[:, 0]))[:, None]
    q = e / total
    log_q = torch.where(live, t - high - torch.log(total), torch.zeros_like(t))

    def grad_of(p):
        g = p.scatter_add(1, at, -q)
        return g * torch.where(some, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]

    z, lse, dx, dw = _head(s, grad_of)
    terms = torch.where(live, q * (log_q - (z.gather(1, at) - lse)), torch.zeros_like(q))
    loss = terms.sum(1)
    return (loss, dx, dw) if s["grad"] else (loss, lse[:, 0])


def run(state):
    s = state
    if not own:
        return {"norm": _norm, "norm_backward": _norm_backward, "loss": _loss,
                "distil": _distil}[s["op"]](s)
    import fp16_gemm_relu_gb300 as tg

    if s["op"] == "norm":
        return tg.layer_norm(s["x"], s["gamma"], s["beta"], eps=EPS, stats=s["stats"])
    if s["op"] == "norm_backward":
        return tg.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"])
    layout = tg.TG_HEAD_VOCAB_MAJOR if s["layout"] == "vocab" else tg.TG_HEAD_WIDTH_MAJOR
    if s["op"] == "loss":
        if not s["grad"]:
            return tg.linear_cross_entropy(s["x"], s["weight"], s["target"],
                                           ignore_index=IGNORE, layout=layout, return_lse=True)
        return tg.linear_cross_entropy_step(s["x"], s["weight"], s["target"], s["dloss"],
                                            ignore_index=IGNORE, layout=layout)
    if not s["grad"]:
        return tg.linear_distillation(s["x"], s["weight"], s["index"], s["logits"],
                                      temperature=s["temperature"], layout=layout,
                                      return_lse=True)
    return tg.linear_distillation_step(s["x"], s["weight"], s["index"], s["logits"], s["dloss"],
                                       temperature=s["temperature"], layout=layout)


def work(case):
    rows, width = case["tokens"], case["width"]
    if case["op"] == "norm":
        return {"bytes": 4 * rows * width + 4 * width + (8 * rows if case["stats"] else 0),
                "flops": 8 * rows * width}
    if case["op"] == "norm_backward":
        return {"bytes": 6 * rows * width + 6 * width + 8 * rows, "flops": 14 * rows * width}
    vocab = case["vocab"]
    passes = 3 if case["grad"] else 1  # the logits, and dX and dW
    each = 2 * (rows * width + vocab * width)
    side = 16 * rows  # target, loss and the log sum, or the loss's weight
    if case["op"] == "distil":
        side = 8 * rows + rows * case["top"] * (8 + (2 if case["teacher"] == "float16" else 4))
    return {"bytes": each * (2 if case["grad"] else 1) + side,
            "flops": 2 * rows * vocab * width * passes}


def exact(case, seed):
    if work(case)["flops"] > EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    d = torch.float64
    x = s["x"].to(d)
    if case["op"] == "norm":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = (x - mean[:, None]) * rstd[:, None] * s["gamma"].to(d) + s["beta"].to(d)
        return (y, mean, rstd) if case["stats"] else y
    if case["op"] == "norm_backward":
        dy, gamma = s["dy"].to(d), s["gamma"].to(d)
        rstd = s["rstd"].to(d)[:, None]
        hat = (x - s["mean"].to(d)[:, None]) * rstd
        g = gamma * dy
        dx = rstd * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
        return dx, torch.einsum("tn,tn->n", dy, hat), dy.sum(0)
    w = s["weight"].to(d)
    if case["layout"] == "width":
        w = w.t()
    tau = float(case.get("temperature", 1.0))
    rows, vocab = case["tokens"], case["vocab"]
    loss, lse = (torch.zeros(rows, dtype=d, device=x.device) for _ in range(2))
    if case["grad"]:
        dx, dw = torch.zeros_like(x), torch.zeros(vocab, case["width"], dtype=d, device=x.device)
    for t0 in range(0, rows, 1024):
        t1 = min(rows, t0 + 1024)
        z = torch.mm(x[t0:t1], w.t()) / tau
        lse[t0:t1] = torch.logsumexp(z, dim=1)
        logp = z.sub_(lse[t0:t1, None])
        if case["op"] == "loss":
            keep = s["target"][t0:t1] != IGNORE
            q = keep[:, None].to(d)
            index = s["target"][t0:t1].clamp_min(0)[:, None]
            entropy = torch.zeros_like(loss[t0:t1])
        else:
            valid = s["index"][t0:t1] >= 0
            keep = valid.any(1)
            teacher = (s["logits"][t0:t1].to(d) / tau).masked_fill(~valid, -1e300)
            q = torch.softmax(teacher, dim=1) * keep[:, None]
            index = s["index"][t0:t1].clamp_min(0)
            entropy = torch.special.entr(q).sum(1)
        loss[t0:t1] = -entropy - (q * torch.take_along_dim(logp, index, 1)).sum(1)
        if case["grad"]:
            g = logp.exp_()
            g.mul_(keep[:, None])
            g.scatter_add_(1, index, -q)
            g.mul_(s["dloss"][t0:t1, None].to(d) / tau)
            dx[t0:t1] = torch.mm(g, w)
            dw.addmm_(g.t(), x[t0:t1])
    if not case["grad"]:
        return loss, lse
    return loss, dx, dw if case["layout"] == "vocab" else dw.t().contiguous()
