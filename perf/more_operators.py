"""The operators of a fine-tuning step, as measured workloads: the gated feed-forward product with its
gradients, preference and policy losses of a linear head with theirs, and the unscaling and clipping of
all gradients by their global norm.

Each case is one call that such a step, or a model that answers, makes on the inputs that it has in
hand.  ``run`` computes it from elementary torch operations in 32 bits (rounded once at the end), or,
where ``own`` is true, through this package's entry points.  ``exact`` is the same from the definitions
in 64 bits.

Layouts: activations are (tokens, width) fp16 rows; the weights of the gated product are (width, hidden),
as the framework's GEMM takes its right operand, or (hidden, width); a head's weight is (vocab, width) or
(width, vocab).  Log probabilities, advantages, losses and norms are float32.
"""

import math

import torch

own = False

IGNORE = -100
LOSS_SCALE = 8192.0  # fp16 training scales the loss so that the gradients stay normal numbers
BETA = 0.1           # weight of a preference's log ratios
CLIP = (0.2, 0.28)   # how far a policy's ratio counts below and above 1
EXACT_FLOPS = 1.2e13  # 64-bit products beyond this take too long on this GPU


def listed():
    return [
        # the feed-forward block of a model that answers one request, token by token
        dict(name="gated, one token", op="gated", tokens=1, width=4096, hidden=14336, pad=0,
             act="silu", trans=False, keep=False),
        # 64 requests at once: both weights are read once
        dict(name="gated, 64 requests", op="gated", tokens=64, width=8192, hidden=28672, pad=0,
             act="silu", trans=True, keep=False),
        # a training step's forward pass of a block, pre-activations kept for the backward pass
        dict(name="gated, training", op="gated", tokens=8192, width=4096, hidden=14336, pad=0,
             act="silu", trans=False, keep=True),
        # sizes that are multiples of nothing: every row starts unaligned
        dict(name="gated, ragged", op="gated", tokens=1023, width=2047, hidden=5461, pad=3,
             act="gelu_tanh", trans=False, keep=True),
        # the backward pass of that training step
        dict(name="gated backward, training", op="gated_backward", tokens=8192, width=4096,
             hidden=14336, pad=0, act="silu", trans=False),
        # a short batch through a small block of odd sizes
        dict(name="gated backward, ragged", op="gated_backward", tokens=509, width=1023, hidden=4095,
             pad=5, act="relu", trans=True),
        # a few pairs of short answers on a small model
        dict(name="preference, small batch", op="preference", pairs=4, tokens=256, vocab=28672,
             width=1024, layout="vocab", smoothing=0.0, average=False, grad=True),
        # a preference step on a ragged vocabulary, labels smoothed
        dict(name="preference, training", op="preference", pairs=16, tokens=4096, vocab=65537,
             width=2048, layout="vocab", smoothing=0.1, average=False, grad=True),
        # a clipped policy step with its penalty against a reference, the largest case
        dict(name="policy, training", op="policy", tokens=4096, vocab=131072, width=2048,
             layout="vocab", kl=0.04, grad=True),
        # how far a policy has moved on a held-out batch; the head stored as the GEMM's operand
        dict(name="policy, evaluation", op="policy", tokens=2048, vocab=28672, width=4096,
             layout="width", kl=0.04, grad=False),
        # the gradients of a small model: latency alone
        dict(name="clip, small model", op="clip", layers=2, width=256, hidden=512, vocab=1000,
             ratio=0.5),
        # the gradients of a model of 1.3 billion weights
        dict(name="clip, large model", op="clip", layers=12, width=4096, hidden=8192, vocab=28672,
             ratio=0.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):  # most models' sizes are multiples of 8, some are not
    n = _log(rng, lo, hi)
    return max(lo, n // 8 * 8) if rng.random() < 0.7 else n


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_backward", "gated_backward", "preference", "policy",
                     "clip"])
    if op in ("gated", "gated_backward"):
        while True:
            tokens, width, hidden = _log(rng, 1, 16384), _size(rng, 64, 8192), _size(rng, 64, 28672)
            if tokens * width * hidden <= 8192 * 4096 * 14336 and tokens * hidden <= 8192 * 28672:
                break
        case = dict(op=op, tokens=tokens, width=width, hidden=hidden, pad=rng.choice([0, 0, 8, 3]),
                    act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu", "none"]),
                    trans=rng.random() < 0.5)
        if op == "gated":
            case["keep"] = rng.random() < 0.5
        return case
    if op == "clip":
        while True:
            layers, width = _log(rng, 1, 12), _size(rng, 64, 4096)
            hidden, vocab = _size(rng, 64, 16384), _log(rng, 100, 131072)
            if layers * 3 * width * hidden + vocab * width <= 1_300_000_000:
                break
        return dict(op=op, layers=layers, width=width, hidden=hidden, vocab=vocab,
                    ratio=rng.choice([0.1, 0.5, 2.0]))
    while True:
        tokens, vocab, width = _log(rng, 2, 8192), _log(rng, 1000, 131072), _size(rng, 64, 8192)
        if tokens * vocab * width <= 4096 * 65537 * 2048 and tokens * vocab <= 4096 * 131072:
            break
    case = dict(op=op, tokens=tokens, vocab=vocab, width=width,
                layout=rng.choice(["vocab", "vocab", "width"]), grad=rng.random() < 0.7)
    if op == "preference":
        case.update(pairs=_log(rng, 1, max(1, min(64, tokens // 2))), smoothing=rng.choice([0.0, 0.1]),
                    average=rng.random() < 0.3)
    else:
        case["kl"] = rng.choice([0.0, 0.04, 0.1])
    return case


def _shapes(case):
    """The weights of a model: per block a norm's two vectors and three matrices, then the head."""
    width, hidden = case["width"], case["hidden"]
    block = [(width,), (width,), (width, hidden), (width, hidden), (hidden, width)]
    return block * case["layers"] + [(case["vocab"], width)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device=dev, dtype=torch.float32)

    def matrix(rows, cols, scale, pad=0):  # the columns [0, cols) of a buffer of cols + pad
        buf = torch.zeros(rows, cols + pad, dtype=torch.float16, device=dev)
        for r0 in range(0, rows, 16384):  # in pieces: 32-bit normals of the whole are large
            r1 = min(rows, r0 + 16384)
            buf[r0:r1, :cols] = normal(r1 - r0, cols) * scale
        return buf[:, :cols]

    state = dict(case)
    if case["op"] == "clip":
        # gradients under the loss scale: each weight's of its own size; a norm's vectors are float32
        grads = []
        for shape in _shapes(case):
            size = LOSS_SCALE * 2e-5 * float(torch.exp(normal(1)).clamp_(0.2, 5.0))
            g = torch.empty(shape, device=dev, dtype=torch.float32 if len(shape) == 1 else torch.float16)
            flat = g.view(-1)
            for i in range(0, flat.numel(), 1 << 26):
                j = min(flat.numel(), i + (1 << 26))
                flat[i:j] = normal(j - i) * size
            grads.append(g)
        state["grads"] = grads
        squares = sum(float(g.double().square().sum()) if g.numel() < 1 << 24
                      else sum(float(p.float().square().sum()) for p in g.view(-1).split(1 << 26))
                      for g in grads)
        state["max_norm"] = case["ratio"] * math.sqrt(squares) / LOSS_SCALE
        return state
    tokens, width = case["tokens"], case["width"]
    if case["op"] in ("gated", "gated_backward"):
        hidden, pad = case["hidden"], case["pad"]
        x = matrix(tokens, width, 1.0, pad)  # a normalised stream
        # pre-activations of a few units: gates from closed to open
        w_gate, w_up = (matrix(*((hidden, width) if case["trans"] else (width, hidden)),
                               1.5 / math.sqrt(width), pad) for _ in range(2))
        state.update(x=x, w_gate=w_gate, w_up=w_up)
        if case["op"] == "gated_backward":
            state["dh"] = matrix(tokens, hidden, 0.25, pad)
            for name, w in (("gate", w_gate), ("up", w_up)):  # what the forward pass kept
                wf = w.float().t() if case["trans"] else w.float()
                state[name] = (x.float() @ wf).half()
        return state
    vocab = case["vocab"]
    x = normal(tokens, width).half()
    weight = matrix(vocab, width, 2.0 / math.sqrt(width))
    # a text's tokens: frequent ones have low numbers; a prompt's tokens do not count
    u = uniform(tokens)
    target = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)
    target[uniform(tokens) < (0.2 if tokens > 8 else 0.0)] = IGNORE
    live = target != IGNORE
    logp = torch.zeros(tokens, device=dev)
    for t0 in range(0, tokens, 1024):
        t1 = min(tokens, t0 + 1024)
        z = x[t0:t1].float() @ weight.t().float()
        at = target[t0:t1].clamp_min(0)[:, None]
        logp[t0:t1] = (z.gather(1, at) - torch.logsumexp(z, 1, keepdim=True))[:, 0]
    state.update(x=x, weight=weight if case["layout"] == "vocab" else weight.t().contiguous(),
                 target=target, reference=logp + 0.1 * normal(tokens))
    if case["op"] == "preference":
        # answers of all lengths, some empty; the rows behind the last are a batch's padding
        pairs = case["pairs"]
        cuts = (uniform(2 * pairs) * (tokens + 1)).long().clamp_(0, tokens).sort().values
        offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), cuts])
        # the model already prefers most chosen answers by a few nats over the reference
        ahead = torch.stack([uniform(pairs) * 12 - 4, uniform(pairs) * 12 - 8], 1).view(-1)
        ahead = torch.cat([ahead * (2 * pairs / tokens), torch.zeros(1, device=dev)])
        sequence = torch.searchsorted(offsets, torch.arange(tokens, device=dev), right=True) - 1
        state["offsets"], state["reference"] = offsets, state["reference"] - ahead[sequence]
        if case["grad"]:
            state["dloss"] = torch.full((pairs,), LOSS_SCALE / pairs, device=dev)
        return state
    # the policy has moved a little since its tokens were drawn; no ratio lies on a border of the
    # clipping, where either gradient is right
    moved = 0.2 * normal(tokens)
    for border in (math.log(1 - CLIP[0]), math.log(1 + CLIP[1])):
        near = (moved - border).abs() < 0.005
        moved = torch.where(near, moved + 0.02, moved)
    state["old"] = logp - moved
    state["advantage"] = normal(tokens)
    if case["grad"]:
        state["dloss"] = torch.full((tokens,), LOSS_SCALE, device=dev) / live.sum().clamp_min(1)
    return state


def _activation(v, act):
    """act(v) and its derivative."""
    if act == "none":
        return v, torch.ones_like(v)
    if act == "relu":
        on = (v > 0).to(v.dtype)
        return v * on, on
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-v))
        return v * s, s * (1.0 + v * (1.0 - s))
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5)))
        return v * cdf, cdf + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (v + 0.044715 * v * v * v))
    slope = 0.5 * (1.0 + t) + 0.5 * v * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * v * v)
    return 0.5 * v * (1.0 + t), slope


def _gated(s):
    x = s["x"].float()
    wg, wu = s["w_gate"].float(), s["w_up"].float()
    gate, up = (x @ wg.t(), x @ wu.t()) if s["trans"] else (x @ wg, x @ wu)
    h = (_activation(gate, s["act"])[0] * up).half()
    return (h, gate.half(), up.half()) if s["keep"] else h


def _gated_backward(s):
    x, dh = s["x"].float(), s["dh"].float()
    wg, wu = s["w_gate"].float(), s["w_up"].float()
    value, slope = _activation(s["gate"].float(), s["act"])
    dg, du = dh * s["up"].float() * slope, dh * value
    if s["trans"]:
        return (dg @ wg + du @ wu).half(), (dg.t() @ x).half(), (du.t() @ x).half()
    return (dg @ wg.t() + du @ wu.t()).half(), (x.t() @ dg).half(), (x.t() @ du).half()


def _logits(s):
    """Logits, the targets' log probabilities (0 for a row that does not count), and what gives dX and dW
    from each row's d total / d log probability."""
    x, w = s["x"].float(), s["weight"].float()
    by_vocab = s["layout"] == "vocab"
    z = x @ (w.t() if by_vocab else w)
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    live = s["target"] != IGNORE
    at = torch.where(live, s["target"], torch.zeros_like(s["target"]))[:, None]
    logp = (z.gather(1, at) - top - torch.log(total))[:, 0]
    logp = torch.where(live, logp, torch.zeros_like(logp))

    def gradients(slope):
        g = (e / total).scatter_add(1, at, torch.full_like(at, -1.0, dtype=torch.float32))
        g = g * torch.where(live, -slope, torch.zeros_like(slope))[:, None]
        return ((g @ (w if by_vocab else w.t())).half(),
                (g.t() @ x if by_vocab else x.t() @ g).half())

    return live, logp, gradients


def _preference(s):
    live, logp, gradients = _logits(s)
    pairs, offsets = s["pairs"], s["offsets"]
    rows = torch.arange(s["tokens"], device=logp.device)
    inside = (rows[:, None] >= offsets[:-1]) & (rows[:, None] < offsets[1:]) & live[:, None]
    ratio = torch.where(live, logp - s["reference"], torch.zeros_like(logp))
    sums = (ratio[:, None].double() * inside).sum(0)
    count = inside.sum(0).clamp_min(1).double() if s["average"] else torch.ones_like(sums)
    ratios = (sums / count).view(pairs, 2)
    margin = BETA * (ratios[:, 0] - ratios[:, 1])
    smooth = s["smoothing"]

    def log_sigmoid(v):
        return -(torch.log(1.0 + torch.exp(-v.abs())) + (-v).clamp_min(0.0))

    loss = -(1.0 - smooth) * log_sigmoid(margin) - smooth * log_sigmoid(-margin)
    if not s["grad"]:
        return loss.float(), ratios.float()
    slope = BETA * (smooth - 1.0 / (1.0 + torch.exp(margin)))  # d loss / d ratio of the chosen
    slope = slope * s["dloss"]
    per_sequence = torch.stack([slope, -slope], 1).view(-1) / count
    dx, dw = gradients((inside.double() * per_sequence).sum(1).float())
    return loss.float(), ratios.float(), dx, dw


def _policy(s):
    live, logp, gradients = _logits(s)
    adv, kl = s["advantage"], s["kl"]
    ratio = torch.exp(logp - s["old"])
    kept = torch.minimum(torch.maximum(ratio, torch.full_like(ratio, 1.0 - CLIP[0])),
                         torch.full_like(ratio, 1.0 + CLIP[1]))
    loss = -torch.minimum(ratio * adv, kept * adv)
    slope = torch.where(ratio * adv <= kept * adv, -adv * ratio, torch.zeros_like(ratio))
    if kl:
        d = s["reference"] - logp
        loss = loss + kl * (torch.exp(d) - d - 1.0)
        slope = slope + kl * (1.0 - torch.exp(d))
    zero = torch.zeros_like(loss)
    loss = torch.where(live, loss, zero)
    if not s["grad"]:
        return loss, logp
    dx, dw = gradients(slope * s["dloss"])
    return loss, logp, dx, dw


def _clip(s):
    total = torch.zeros((), device="cuda", dtype=torch.float64)
    for g in s["grads"]:
        total = total + g.float().square().sum().double()
    norm = torch.sqrt(total) / LOSS_SCALE
    factor = (torch.clamp(s["max_norm"] / norm, max=1.0) / LOSS_SCALE).float()
    return [norm.float()] + [g.float() * factor for g in s["grads"]]


def run(state):
    s = state
    if not own:
        return {"gated": _gated, "gated_backward": _gated_backward, "preference": _preference,
                "policy": _policy, "clip": _clip}[s["op"]](s)
    import fp16_gemm_relu_gb300 as tg

    if s["op"] in ("gated", "gated_backward"):
        act = {"none": tg.TG_ACT_NONE, "relu": tg.TG_ACT_RELU, "gelu": tg.TG_ACT_GELU,
               "gelu_tanh": tg.TG_ACT_GELU_TANH, "silu": tg.TG_ACT_SILU}[s["act"]]
        if s["op"] == "gated":
            return tg.gated_linear(s["x"], s["w_gate"], s["w_up"], activation=act,
                                   trans_w=s["trans"], keep=s["keep"])
        return tg.gated_linear_backward(s["dh"], s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"],
                                        activation=act, trans_w=s["trans"])
    if s["op"] == "clip":
        norm, grads = tg.clip_gradients(s["grads"], s["max_norm"], loss_scale=LOSS_SCALE)
        return [norm] + grads
    layout = tg.TG_HEAD_VOCAB_MAJOR if s["layout"] == "vocab" else tg.TG_HEAD_WIDTH_MAJOR
    if s["op"] == "preference":
        options = dict(reference=s["reference"], beta=BETA, label_smoothing=s["smoothing"],
                       average=s["average"], ignore_index=IGNORE, layout=layout)
        if not s["grad"]:
            return tg.linear_preference(s["x"], s["weight"], s["target"], s["offsets"], **options)
        return tg.linear_preference_step(s["x"], s["weight"], s["target"], s["offsets"], s["dloss"],
                                         **options)
    options = dict(reference=s["reference"] if s["kl"] else None, kl_weight=s["kl"],
                   clip_low=CLIP[0], clip_high=CLIP[1], ignore_index=IGNORE, layout=layout)
    if not s["grad"]:
        return tg.linear_policy(s["x"], s["weight"], s["target"], s["old"], s["advantage"], **options)
    return tg.linear_policy_step(s["x"], s["weight"], s["target"], s["old"], s["advantage"],
                                 s["dloss"], **options)


def work(case):
    if case["op"] == "clip":
        vectors = sum(math.prod(n) for n in _shapes(case) if len(n) == 1)
        matrices = sum(math.prod(n) for n in _shapes(case) if len(n) == 2)
        return {"bytes": 8 * vectors + 6 * matrices, "flops": 3 * (vectors + matrices)}
    tokens, width = case["tokens"], case["width"]
    if case["op"] in ("gated", "gated_backward"):
        hidden = case["hidden"]
        x, w, h = 2 * tokens * width, 2 * width * hidden, 2 * tokens * hidden
        if case["op"] == "gated":
            return {"bytes": x + 2 * w + (3 if case["keep"] else 1) * h,
                    "flops": 4 * tokens * width * hidden}
        return {"bytes": 2 * x + 4 * w + 3 * h, "flops": 8 * tokens * width * hidden}
    vocab = case["vocab"]
    each = 2 * (tokens * width + vocab * width)
    side = 32 * tokens  # targets, log probabilities, advantages, losses
    return {"bytes": each * (2 if case["grad"] else 1) + side,
            "flops": 2 * tokens * vocab * width * (3 if case["grad"] else 1)}


def _act64(v, act):
    """act(v) and its derivative, by automatic differentiation of the definition."""
    v = v.detach().requires_grad_(True)
    f = torch.nn.functional
    with torch.enable_grad():
        y = {"none": lambda: v * 1.0, "relu": lambda: f.relu(v), "silu": lambda: f.silu(v),
             "gelu": lambda: f.gelu(v), "gelu_tanh": lambda: f.gelu(v, approximate="tanh")}[act]()
        slope, = torch.autograd.grad(y.sum(), v)
    return y.detach(), slope


def exact(case, seed):
    if work(case)["flops"] > EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "clip":
        norm = math.sqrt(sum(float(torch.linalg.vector_norm(g, dtype=d)) ** 2 for g in s["grads"]))
        norm /= LOSS_SCALE
        factor = min(1.0, s["max_norm"] / norm) / LOSS_SCALE
        return [torch.tensor(norm, dtype=d, device="cuda")] + [g.to(d) * factor for g in s["grads"]]
    x = s["x"].to(d)
    if case["op"] in ("gated", "gated_backward"):
        wg, wu = (w.to(d).t() if case["trans"] else w.to(d) for w in (s["w_gate"], s["w_up"]))
        if case["op"] == "gated":
            gate, up = torch.mm(x, wg), torch.mm(x, wu)
            h = _act64(gate, case["act"])[0] * up
            return (h, gate, up) if case["keep"] else h
        value, slope = _act64(s["gate"].to(d), case["act"])
        dh = s["dh"].to(d)
        dg, du = slope * s["up"].to(d) * dh, value * dh
        dwg, dwu = torch.mm(x.t(), dg), torch.mm(x.t(), du)
        dx = torch.mm(dg, wg.t()) + torch.mm(du, wu.t())
        return (dx, dwg.t(), dwu.t()) if case["trans"] else (dx, dwg, dwu)
    w = s["weight"].to(d) if case["layout"] == "vocab" else s["weight"].to(d).t()
    tokens = case["tokens"]
    keep = s["target"] != IGNORE
    index = s["target"].clamp_min(0)[:, None]
    logp = torch.zeros(tokens, dtype=d, device=x.device)
    for t0 in range(0, tokens, 1024):
        t1 = min(tokens, t0 + 1024)
        rows = torch.log_softmax(torch.mm(x[t0:t1], w.t()), dim=1)
        logp[t0:t1] = torch.take_along_dim(rows, index[t0:t1], 1)[:, 0]
    logp = (logp * keep).requires_grad_(True)
    with torch.enable_grad():  # the loss from the log probabilities, differentiated by torch
        if case["op"] == "preference":
            at = s["offsets"].tolist()
            ratios = []
            for a, b in zip(at[:-1], at[1:]):
                kept = ((logp - s["reference"].to(d)) * keep)[a:b]
                ratios.append(kept.sum() / (max(int(keep[a:b].sum()), 1) if case["average"] else 1))
            ratios = torch.stack(ratios).view(-1, 2)
            margin = BETA * (ratios[:, 0] - ratios[:, 1])
            f = torch.nn.functional.logsigmoid
            loss = -(1 - case["smoothing"]) * f(margin) - case["smoothing"] * f(-margin)
            outputs = (loss, ratios)
        else:
            ratio = torch.exp(logp - s["old"].to(d))
            adv = s["advantage"].to(d)
            loss = torch.maximum(-ratio * adv, -ratio.clamp(1 - CLIP[0], 1 + CLIP[1]) * adv)
            if case["kl"]:
                away = s["reference"].to(d) - logp
                loss = loss + case["kl"] * (torch.expm1(away) - away)
            loss = loss * keep
            outputs = (loss, logp)
        if not case["grad"]:
            return tuple(o.detach() for o in outputs)
        slope, = torch.autograd.grad((loss * s["dloss"].to(d)).sum(), logp)
    dx, dw = torch.zeros_like(x), torch.zeros(case["vocab"], case["width"], dtype=d, device=x.device)
    for t0 in range(0, tokens, 1024):
        t1 = min(tokens, t0 + 1024)
        g = torch.softmax(torch.mm(x[t0:t1], w.t()), dim=1)
        g.scatter_add_(1, index[t0:t1], torch.full_like(g[:, :1], -1.0))
        g.mul_(-(slope * keep)[t0:t1, None])
        dx[t0:t1] = torch.mm(g, w)
        dw.addmm_(g.t(), x[t0:t1])
    return (*(o.detach() for o in outputs), dx,
            dw if case["layout"] == "vocab" else dw.t().contiguous())
