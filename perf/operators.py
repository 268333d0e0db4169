"""Measured cases of the operators over rows of logits: log probabilities of
given tokens (with entropy and top alternatives), their gradient, and
distillation from a teacher's top entries (loss, loss with gradient, gradient).

``own = False`` computes every case in its plain form, elementary torch
operations in 32 bits; ``own = True`` makes the calls of the framework.

Notation: z is a row of V logits, tau the temperature, x = z / tau,
lse = log sum exp x, p = exp(x - lse).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NEG_INF = float("-inf")


def _case(name, op, rows, vocab, dtype, **more):
    case = {"name": name, "op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "pad": 0,
            "k": 0, "entropy": False, "temperature": 1.0, "mode": "none", "masked": 0.0,
            "absent": 0.0, "stats": False}
    case.update(more)
    return case


def listed():
    return [
        # Serving, one stream: the new token's log probability with the 20
        # alternatives an API reports beside it.
        _case("logprobs_one_token", "logprobs", 1, 131072, "bf16", k=20),
        # Serving, a batch of streams with a small report and the entropy a
        # sampler watches; some rows constrained to a grammar's tokens.
        _case("logprobs_batch", "logprobs", 64, 32768, "f16", k=5, entropy=True, masked=0.25),
        # A large classifier head (21,843 classes, odd) over a batch of images,
        # the 32 best classes each.
        _case("logprobs_classes", "logprobs", 300, 21843, "f32", k=32),
        # Scoring a prompt: every position's token with its alternatives, an
        # odd vocabulary in rows padded for a product's tiles, cooled.
        _case("logprobs_prompt_top", "logprobs", 2048, 50001, "bf16", pad=47, k=20,
              temperature=0.7),
        # Scoring samples for policy training: log probability and entropy of
        # every position and the statistics its backward pass wants, the
        # largest case.
        _case("logprobs_score", "logprobs", 4096, 131072, "bf16", entropy=True, absent=0.1,
              stats=True),
        # The gradient of that training step, from the forward's statistics.
        _case("logprobs_grad", "logprobs_grad", 4096, 65536, "bf16", entropy=True, absent=0.1),
        # The same of a smaller odd batch, with gradients of the alternatives
        # too.
        _case("logprobs_grad_odd", "logprobs_grad", 255, 50001, "f16", k=8, temperature=1.3),
        # Evaluating a small student on a 1,000-class teacher.
        _case("distill_eval_classes", "distill", 16, 1000, "f32", k=5, mode="renorm"),
        # Evaluating a student: the loss alone, unlisted tokens as one event.
        _case("distill_eval", "distill", 1024, 131072, "bf16", k=32, mode="tail"),
        # A training step: the loss and its gradient, ordinary size.
        _case("distill_step_odd", "distill_step", 777, 50001, "f32", k=20, mode="renorm",
              temperature=2.0, absent=0.1),
        # A training step of a long batch, 64 teacher entries.
        _case("distill_step", "distill_step", 2048, 131072, "bf16", k=64, mode="tail",
              absent=0.1),
        # The gradient alone, where the loss's weight was not known before.
        _case("distill_grad", "distill_grad", 2048, 65536, "f16", k=32, mode="tail"),
    ]


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_grad", "distill", "distill_step",
                     "distill_grad"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    rows = int(round(math.exp(rng.uniform(0.0, math.log(4096)))))
    vocab = int(round(math.exp(rng.uniform(math.log(500), math.log(200000)))))
    vocab = max(500, min(vocab, 2 ** 27 // rows))
    more = {"stats": rng.random() < 0.5,
            "pad": rng.choice([0, 0, 1, 3, 24, 101]),
            "temperature": rng.choice([1.0, 1.0, round(rng.uniform(0.5, 2.0), 2)]),
            "absent": rng.choice([0.0, 0.2])}
    if op.startswith("logprobs"):
        more.update(k=rng.choice([0, 1, rng.randint(2, 32)]), entropy=rng.random() < 0.5,
                    masked=rng.choice([0.0, 0.0, 0.3]))
        more["stats"] = more["stats"] and op == "logprobs"
    else:
        more["stats"] = False
        more.update(k=rng.choice([1, rng.randint(2, 32), rng.randint(33, 128)]),
                    mode=rng.choice(["renorm", "tail"]))
    case = _case("drawn", op, rows, vocab, dtype, **more)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# Inputs: what a user's program holds before the call.


def _weight(case):
    """Per-row weight of a mean over the rows; half-precision training scales
    its loss so that gradients stay clear of the type's smallest values."""
    return (16384.0 if case["dtype"] == "f16" else 1.0) / case["rows"]


def _inputs(case, seed):
    """Logits of varying sharpness, a row buffer with `pad` unused columns,
    and the operator's other inputs, from the seed alone."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rows, vocab, k = case["rows"], case["vocab"], case["k"]
    dtype = DTYPES[case["dtype"]]
    buffer = torch.zeros((rows, vocab + case["pad"]), dtype=dtype, device=dev)
    logits = buffer[:, :vocab]
    step = max(1, 2 ** 27 // vocab)
    teacher = torch.zeros((rows, k, 2), dtype=torch.int32, device=dev)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        z = torch.randn((n, vocab), device=dev, generator=gen)
        z *= 1.0 + 2.0 * torch.rand((n, 1), device=dev, generator=gen)
        # Six tokens the context points at, apart from the bulk.
        hot = torch.randint(vocab, (n, 6), device=dev, generator=gen)
        z.scatter_add_(1, hot, 8.0 * torch.rand((n, 6), device=dev, generator=gen))
        if case["masked"]:
            free = torch.rand((n, vocab), device=dev, generator=gen) < 0.01
            free[:, :1] = True
            held = torch.rand((n, 1), device=dev, generator=gen) < case["masked"]
            z = torch.where(held & ~free, torch.full_like(z, NEG_INF), z)
        logits[r:r + n] = z.to(dtype)
        if case["op"].startswith("distill"):
            # A teacher that mostly agrees: its own noise on the same logits.
            y = z + 0.7 * torch.randn((n, vocab), device=dev, generator=gen)
            best, index = torch.topk(y, k, dim=1)
            value = best - torch.logsumexp(y, 1, keepdim=True)
            teacher[r:r + n, :, 0] = value.contiguous().view(torch.int32)
            teacher[r:r + n, :, 1] = index.to(torch.int32)
        del z
    state = {"case": case, "buffer": buffer, "logits": logits}
    if case["op"].startswith("distill"):
        if case["absent"]:
            # Shorter lists: the last half of some rows' entries is absent.
            gone = torch.rand((rows, 1), device=dev, generator=gen) < case["absent"]
            gone = gone & (torch.arange(k, device=dev) >= (k + 1) // 2)
            teacher[:, :, 1] = torch.where(gone, torch.full_like(teacher[:, :, 1], -1),
                                           teacher[:, :, 1])
        state["teacher"] = teacher
        state["grad_loss"] = torch.rand((rows,), device=dev, generator=gen) * _weight(case)
    else:
        targets = torch.randint(vocab, (rows,), device=dev, generator=gen, dtype=torch.int32)
        likely = torch.argmax(logits, 1).to(torch.int32)
        targets = torch.where(torch.rand((rows,), device=dev, generator=gen) < 0.5, likely,
                              targets)
        # Padded positions ask for no token.
        none = torch.rand((rows,), device=dev, generator=gen) < case["absent"]
        state["targets"] = torch.where(none, torch.full_like(targets, -1), targets)
    return state, gen


def _stats64(logits, tau, listed=None, step=2 ** 26):
    """Row maximum, log sum, entropy and (with `listed`) the log probability of
    the tokens not listed, in 64 bits."""
    rows, vocab = logits.shape
    parts = []
    n = max(1, step // vocab)
    for r in range(0, rows, n):
        z = logits[r:r + n].double()
        top = z.amax(1, keepdim=True)
        d = (z - top) / tau
        e = torch.exp(d)
        total = e.sum(1)
        logsum = torch.log(total)
        entropy = logsum - torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1) / total
        tail = torch.zeros_like(logsum)
        if listed is not None:
            tail = torch.logsumexp(d.masked_fill(_mask(listed[r:r + n], vocab), NEG_INF), 1) - logsum
        parts.append(torch.stack([top[:, 0], logsum, entropy, tail]))
    return torch.cat(parts, 1)


def _mask(ids, vocab):
    """True where a token is listed; absent entries (-1) list none."""
    hit = torch.zeros((ids.shape[0], vocab + 1), dtype=torch.bool, device=ids.device)
    at = torch.where(ids < 0, torch.full_like(ids, vocab), ids).long()
    return hit.scatter_(1, at, True)[:, :vocab]


def prepare(case, seed):
    state, gen = _inputs(case, seed)
    logits = state["logits"]
    rows, vocab, k = case["rows"], case["vocab"], case["k"]
    if case["op"] == "logprobs_grad":
        found = _stats64(logits, case["temperature"]).float()
        state["stats"] = found[:2].t().contiguous()
        state["entropy"] = found[2].contiguous()
        dev = logits.device
        state["grad_logprob"] = torch.randn((rows,), device=dev, generator=gen) * _weight(case)
        state["grad_entropy"] = torch.full((rows,), -0.01 * _weight(case), device=dev)
        if k:
            top = torch.zeros((rows, k, 2), dtype=torch.int32, device=dev)
            top[:, :, 1] = _best(logits, k)
            state["top"] = top
            state["grad_top"] = torch.randn((rows, k), device=dev, generator=gen) * _weight(case)
    elif case["op"] == "distill_grad":
        found = _stats64(logits, case["temperature"], state["teacher"][:, :, 1]).float()
        state["stats"] = found[:2].t().contiguous()
        state["tail"] = found[3].contiguous()
    return state


# ---------------------------------------------------------------------------
# One pass.


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    op = case["op"]
    if op == "logprobs":
        return _plain_logprobs(state)
    if op == "logprobs_grad":
        return _plain_logprobs_grad(state)
    if op == "distill_grad":
        return _plain_distill_grad(state)
    return _plain_distill(state, op == "distill_step")


def _best(logits, k):
    """Indices of the k best logits of each row, equal ones by the lower
    index: distinct 64-bit keys, the value's order above the index's."""
    bits = (logits.float() + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, ~bits + (-2 ** 31), bits)
    key = order * 2 ** 31 + (2 ** 31 - 1 - torch.arange(logits.shape[1], device=logits.device))
    return (2 ** 31 - 1 - torch.topk(key, k, dim=1).values % 2 ** 31).to(torch.int32)


def _plain_logprobs(state):
    case = state["case"]
    z = state["logits"]
    x = z.float() / case["temperature"]
    d = x - x.amax(1, keepdim=True)
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    logp = d - torch.log(total)
    targets = state["targets"].long()
    got = logp.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    out = {"logprob": torch.where(targets < 0, torch.zeros_like(got), got)}
    if case["entropy"]:
        p = e / total
        out["entropy"] = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(1)
    if case["stats"]:
        raw = z.float().amax(1)
        out["stats"] = torch.stack([raw, torch.log(total)[:, 0]], 1)
    if case["k"]:
        out["top_id"] = _best(z, case["k"])
        out["top_logprob"] = logp.gather(1, out["top_id"].long())
    return out


def _plain_logprobs_grad(state):
    case = state["case"]
    tau = case["temperature"]
    z = state["logits"].float()
    targets = state["targets"].long()
    logp = (z - state["stats"][:, :1]) / tau - state["stats"][:, 1:]
    p = torch.exp(logp)
    g = torch.where(targets < 0, torch.zeros_like(state["grad_logprob"]), state["grad_logprob"])
    whole = g[:, None]
    if case["k"]:
        whole = whole + state["grad_top"].sum(1, keepdim=True)
    dz = -whole * p
    if case["entropy"]:
        bend = torch.where(p > 0, p * (logp + state["entropy"][:, None]), torch.zeros_like(p))
        dz = dz - state["grad_entropy"][:, None] * bend
    dz.scatter_add_(1, targets.clamp(min=0)[:, None], g[:, None])
    if case["k"]:
        dz.scatter_add_(1, state["top"][:, :, 1].long(), state["grad_top"])
    return (dz / tau).to(state["logits"].dtype)


def _teacher(state, dtype=torch.float32):
    """The teacher's ids (clamped), which are present, log q, q and q of the
    unlisted tokens (a difference near zero: in 64 bits)."""
    teacher = state["teacher"]
    ids = teacher[:, :, 1].long()
    there = ids >= 0
    value = teacher[:, :, 0].contiguous().view(torch.float32).double()
    value = value.masked_fill(~there, NEG_INF)
    if state["case"]["mode"] == "renorm":
        value = value - torch.logsumexp(value, 1, keepdim=True)
        rest = torch.zeros_like(value[:, 0])
    else:
        rest = (1.0 - torch.exp(value).sum(1)).clamp(min=0.0)
    return ids.clamp(min=0), there, value.to(dtype), torch.exp(value).to(dtype), rest.to(dtype)


def _plain_distill(state, step):
    case = state["case"]
    x = state["logits"].float() / case["temperature"]
    d = x - x.amax(1, keepdim=True)
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    logsum = torch.log(total)
    ids, there, logq, q, rest = _teacher(state)
    zero = torch.zeros_like(q)
    loss = torch.where(q > 0, q * (logq - (d.gather(1, ids) - logsum)), zero).sum(1)
    factor = torch.ones_like(rest)
    if case["mode"] == "tail":
        hit = _mask(state["teacher"][:, :, 1], case["vocab"])
        far = d.masked_fill(hit, NEG_INF)
        high = far.amax(1, keepdim=True)
        tail = (high + torch.log(torch.exp(far - high).sum(1, keepdim=True)) - logsum)[:, 0]
        loss = loss + torch.where(rest > 0, rest * (torch.log(rest) - tail),
                                  torch.zeros_like(rest))
        factor = 1.0 - rest * torch.exp(-tail)
    out = {"loss": loss}
    if step:
        dz = e / total
        mass = (q.sum(1) + rest)[:, None]
        if case["mode"] == "tail":
            dz = torch.where(hit, mass * dz, factor[:, None] * dz)
        dz.scatter_add_(1, ids, torch.where(there, -q, zero))
        out["grad"] = (dz * (state["grad_loss"][:, None] / case["temperature"])).to(
            state["logits"].dtype)
    return out


def _plain_distill_grad(state):
    case = state["case"]
    tau = case["temperature"]
    z = state["logits"].float()
    ids, there, _, q, rest = _teacher(state)
    dz = torch.exp((z - state["stats"][:, :1]) / tau - state["stats"][:, 1:])
    if case["mode"] == "tail":
        hit = _mask(state["teacher"][:, :, 1], case["vocab"])
        mass = (q.sum(1) + rest)[:, None]
        factor = (1.0 - rest * torch.exp(-state["tail"]))[:, None]
        dz = torch.where(hit, mass * dz, factor * dz)
    dz.scatter_add_(1, ids, torch.where(there, -q, torch.zeros_like(q)))
    return (dz * (state["grad_loss"][:, None] / tau)).to(state["logits"].dtype)


def _run_own(state):
    """The framework's call, its configuration, outputs and workspace bound on
    the state's first pass and run on torch's current stream."""
    if "call" not in state:
        state["call"], state["out"] = _bind(state)
    state["call"].run(torch.cuda.current_stream().cuda_stream)
    return state["out"]


def _bind(state):
    from post_processing_amd import logits as lg
    from post_processing_amd import ws

    case = state["case"]
    op, k = case["op"], case["k"]
    rows, vocab = case["rows"], case["vocab"]
    z = state["logits"]
    dtype = {"f32": ws.DTYPE_F32, "f16": ws.DTYPE_F16, "bf16": ws.DTYPE_BF16}[case["dtype"]]
    shape = lg.make_rows(rows=rows, vocab=vocab, row_stride=vocab + case["pad"], dtype=dtype,
                         temperature=case["temperature"])

    def fresh(*size, dtype=torch.float32):
        return torch.empty(size, dtype=dtype, device=z.device)

    if op == "logprobs":
        logprob = fresh(rows)
        entropy = fresh(rows) if case["entropy"] else None
        top = fresh(rows, k, 2, dtype=torch.int32) if k else None
        stats = fresh(rows, 2) if case["stats"] else None
        call = lg.LogProbs(shape, z, targets=state["targets"], logprob=logprob, entropy=entropy,
                           top_k=k, top=top, stats=stats)
        out = {"logprob": logprob}
        if stats is not None:
            out["stats"] = stats
        if entropy is not None:
            out["entropy"] = entropy
        if k:
            out["top_id"] = top[:, :, 1]
            out["top_logprob"] = top.view(torch.float32)[:, :, 0]
        return call, out
    if op == "logprobs_grad":
        grad = fresh(rows, vocab, dtype=z.dtype)
        more = {}
        if k:
            more = {"top_k": k, "top": state["top"], "grad_top": state["grad_top"]}
        if case["entropy"]:
            more["entropy"] = state["entropy"]
            more["grad_entropy"] = state["grad_entropy"]
        call = lg.LogProbsGrad(shape, z, state["stats"], grad, targets=state["targets"],
                               grad_logprob=state["grad_logprob"], **more)
        return call, grad
    mode = lg.DISTILL_TAIL if case["mode"] == "tail" else lg.DISTILL_RENORM
    if op == "distill_grad":
        grad = fresh(rows, vocab, dtype=z.dtype)
        call = lg.DistillGrad(shape, z, state["teacher"], k, mode, state["stats"],
                              state["grad_loss"], grad,
                              tail=state["tail"] if case["mode"] == "tail" else None)
        return call, grad
    out = {"loss": fresh(rows)}
    more = {}
    if op == "distill_step":
        out["grad"] = fresh(rows, vocab, dtype=z.dtype)
        more = {"grad_loss": state["grad_loss"], "grad_logits": out["grad"]}
    return lg.Distill(shape, z, state["teacher"], k, mode, out["loss"], **more), out


# ---------------------------------------------------------------------------


def work(case):
    """Each logit read once and each output written once; per element the
    difference from the maximum, the scale, the exponential and the sum (two
    more for the entropy), and two for a gradient."""
    rows, k = case["rows"], case["k"]
    cells = rows * case["vocab"]
    size = 4 if case["dtype"] == "f32" else 2
    op = case["op"]
    gradient = op in ("logprobs_grad", "distill_step", "distill_grad")
    moved = cells * size * (2 if gradient else 1) + rows * (8 + 8 * k + (8 if case["stats"] else 0))
    flops = cells * (4 + (2 if case["entropy"] else 0) + (2 if gradient else 0))
    return {"bytes": moved, "flops": flops}


def exact(case, seed):
    """The outputs from the definitions in 64 bits, row block by row block."""
    state = prepare(case, seed)
    rows, vocab, k, tau = case["rows"], case["vocab"], case["k"], case["temperature"]
    blocks = []
    n = max(1, 2 ** 26 // vocab)
    for r in range(0, rows, n):
        part = {key: value[r:r + n] for key, value in state.items()
                if isinstance(value, torch.Tensor)}
        blocks.append(_exact_block(case, part, vocab, k, tau))
    if isinstance(blocks[0], dict):
        return {key: torch.cat([b[key] for b in blocks]) for key in blocks[0]}
    return torch.cat(blocks)


def _exact_block(case, part, vocab, k, tau):
    x = part["logits"].double() / tau
    logp = torch.log_softmax(x, 1)
    p = torch.exp(logp)
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    at = torch.arange(x.shape[0], device=x.device)
    if case["op"].startswith("logprobs"):
        t = part["targets"].long()
        asked = t >= 0
        t = t.clamp(min=0)
        plogp = torch.where(p > 0, p * logp, zero)
        entropy = -plogp.sum(1)
        if case["op"] == "logprobs":
            out = {"logprob": torch.where(asked, logp[at, t], zero)}
            if case["entropy"]:
                out["entropy"] = entropy
            if case["stats"]:
                high = x.amax(1)
                out["stats"] = torch.stack([high * tau, torch.logsumexp(x, 1) - high], 1)
            if k:
                # A stable sort keeps equal values in index order.
                order = torch.sort(part["logits"].double(), dim=1, descending=True, stable=True)[1]
                order = order[:, :k]
                out["top_id"] = order.to(torch.int32)
                out["top_logprob"] = torch.gather(logp, 1, order)
            return out
        g = torch.where(asked, part["grad_logprob"].double(), zero)
        dx = -g[:, None] * p
        dx[at, t] += g
        if k:
            gt = part["grad_top"].double()
            dx -= gt.sum(1, keepdim=True) * p
            dx.scatter_add_(1, part["top"][:, :, 1].long(), gt)
        if case["entropy"]:
            dx -= part["grad_entropy"].double()[:, None] * (plogp + p * entropy[:, None])
        return dx / tau
    ids = part["teacher"][:, :, 1].long()
    there = ids >= 0
    value = part["teacher"][:, :, 0].contiguous().view(torch.float32).double()
    q = torch.where(there, torch.exp(value), zero)
    rest = torch.zeros_like(q[:, 0])
    if case["mode"] == "renorm":
        q = q / q.sum(1, keepdim=True)
    else:
        rest = (1.0 - q.sum(1)).clamp(min=0.0)
    spread = torch.zeros((x.shape[0], vocab + 1), dtype=torch.float64, device=x.device)
    spread.scatter_add_(1, torch.where(there, ids, torch.full_like(ids, vocab)), q)
    spread = spread[:, :vocab]
    outside = ~_mask(part["teacher"][:, :, 1], vocab)
    loss = torch.where(q > 0, q * (torch.log(q) - logp.gather(1, ids.clamp(min=0))), zero).sum(1)
    if case["mode"] == "tail":
        tail = torch.logsumexp(logp.masked_fill(~outside, NEG_INF), 1)
        loss = loss + torch.where(rest > 0, rest * (torch.log(rest) - tail), zero)
    if case["op"] == "distill":
        return {"loss": loss}
    if case["mode"] == "tail":
        # The unlisted tokens share q_tail in proportion to p.
        spread = spread + torch.where(outside, rest[:, None] * p * torch.exp(-tail)[:, None], zero)
    mass = (q.sum(1) + rest)[:, None]
    grad = part["grad_loss"].double()[:, None] / tau * (mass * p - spread)
    return {"loss": loss, "grad": grad} if case["op"] == "distill_step" else grad
