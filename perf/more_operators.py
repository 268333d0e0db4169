"""Measured cases of the operators at a language model's two ends: sampling the
next token from rows of logits, the embedding lookup with scaling and its
gradient, and layer norm forward and backward.

``own = False`` computes every case in its plain form, elementary torch
operations; ``own = True`` makes the calls of the framework.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
NEG_INF = float("-inf")
EPS = 1e-5


def _sample(name, rows, vocab, dtype, keep, **more):
    case = {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype,
            "keep": keep, "masked": 0.0, "pad": 0}
    case.update(more)
    return case


def _embed(name, op, rows, width, vocab, dtype, **more):
    case = {"name": name, "op": op, "rows": rows, "width": width, "vocab": vocab,
            "dtype": dtype, "grad_dtype": dtype, "scale": 1.0, "absent": 0.0, "pad": 0}
    case.update(more)
    return case


def _norm(name, op, rows, width, dtype, **more):
    case = {"name": name, "op": op, "rows": rows, "width": width, "dtype": dtype,
            "weight_dtype": dtype, "pad": 0}
    case.update(more)
    return case


def listed():
    return [
        # Serving one stream: temperature, 50 best, nucleus.
        _sample("sample_one", 1, 131072, "bf16", "top_k_p"),
        # Serving a batch of requests, each with its own settings (greedy ones
        # among them), some held to a grammar's tokens.
        _sample("sample_batch", 64, 32768, "f16", "mixed", masked=0.25),
        # Samples for policy training: the whole distribution at a
        # temperature, an odd vocabulary in rows padded for a product's tiles.
        _sample("sample_rollout", 300, 50001, "f32", "all", pad=15),
        # The same of a large batch of requests with their own settings, the
        # largest.
        _sample("sample_many", 1024, 131072, "bf16", "mixed"),
        # One decoding step of a batch: a token's row each.
        _embed("embed_decode", "embed", 64, 4096, 131072, "bf16", scale=64.0),
        # A training batch's rows, some positions padded.
        _embed("embed_batch", "embed", 16384, 4096, 32768, "bf16", scale=64.0, absent=0.1),
        # Fine-tuning a small model of odd sizes.
        _embed("embed_grad_odd", "embed_grad", 777, 1000, 5003, "f32", absent=0.05),
        # A training batch's gradient, tokens as frequent as in text.
        _embed("embed_grad_batch", "embed_grad", 16384, 4096, 32768, "bf16", scale=64.0,
               absent=0.1),
        # One decoding step before the head.
        _norm("norm_decode", "norm", 64, 4096, "bf16"),
        # A training batch, weights in FP32.
        _norm("norm_batch", "norm", 16384, 4096, "bf16", weight_dtype="f32"),
        # The backward pass of an odd width.
        _norm("norm_grad_odd", "norm_grad", 777, 1001, "f32"),
        # The backward pass of a training batch, the largest.
        _norm("norm_grad_batch", "norm_grad", 16384, 4096, "bf16", weight_dtype="f32"),
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "embed", "embed_grad", "norm", "norm_grad"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    pad = rng.choice([0, 0, 1, 8, 24, 101])
    if op == "sample":
        rows = _spread(rng, 1, 1024)
        vocab = max(500, min(_spread(rng, 500, 200000), 2 ** 26 // rows))
        case = _sample("", rows, vocab, dtype, rng.choice(["all", "top_k_p", "mixed", "mixed"]),
                       masked=rng.choice([0.0, 0.0, 0.3]), pad=pad)
    elif op in ("embed", "embed_grad"):
        width = _spread(rng, 64, 8192)
        rows = min(_spread(rng, 1, 16384), 2 ** 25 // width)
        vocab = max(2, min(_spread(rng, 500, 131072), 2 ** 26 // width))
        case = _embed("", op, rows, width, vocab, dtype, scale=rng.choice([1.0, 0.5, 27.7]),
                      absent=rng.choice([0.0, 0.1]), pad=pad)
        if op == "embed_grad":
            case["grad_dtype"] = rng.choice([dtype, "f32"])
    else:
        width = _spread(rng, 64, 16384)
        rows = min(_spread(rng, 1, 16384), 2 ** 25 // width)
        case = _norm("", op, rows, width, dtype, weight_dtype=rng.choice([dtype, "f32"]), pad=pad)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# Inputs: what a user's program holds before the call.


def _generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _padded(rows, width, pad, dtype):
    """Rows of `width` in a buffer with `pad` unused columns."""
    return torch.zeros((rows, width + pad), dtype=dtype, device="cuda")[:, :width]


def _logits(case, gen):
    """Rows as language models answer: a bulk of unlikely tokens and sixteen
    that the context points at, from nearly certain to undecided."""
    rows, vocab = case["rows"], case["vocab"]
    logits = _padded(rows, vocab, case["pad"], DTYPES[case["dtype"]])
    step = max(1, 2 ** 27 // vocab)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        z = torch.randn((n, vocab), device="cuda", generator=gen)
        z *= 1.0 + 1.5 * torch.rand((n, 1), device="cuda", generator=gen)
        hot = torch.randint(vocab, (n, 16), device="cuda", generator=gen)
        high = 4.0 + 14.0 * torch.rand((n, 1), device="cuda", generator=gen)
        z.scatter_(1, hot, high + 2.0 * torch.randn((n, 16), device="cuda", generator=gen))
        if case["masked"]:
            free = torch.rand((n, vocab), device="cuda", generator=gen) < 0.01
            free[:, :1] = True
            held = torch.rand((n, 1), device="cuda", generator=gen) < case["masked"]
            z = torch.where(held & ~free, torch.full_like(z, NEG_INF), z)
        logits[r:r + n] = z.to(DTYPES[case["dtype"]])
    return logits


def _pick(values, rows, gen):
    at = torch.randint(len(values), (rows,), device="cuda", generator=gen)
    return torch.tensor(values, device="cuda")[at].contiguous()


def _settings(case, gen):
    """Every request's temperature (0: greedy), top-k (0: off), top-p and min-p."""
    rows, keep = case["rows"], case["keep"]
    rand = lambda: torch.rand((rows,), device="cuda", generator=gen)  # noqa: E731
    ones = torch.ones((rows,), device="cuda")
    found = {"temperature": 0.6 + 0.7 * rand(), "top_k": torch.zeros_like(ones).int(),
             "top_p": ones, "min_p": torch.zeros_like(ones)}
    if keep == "top_k_p":
        found["top_k"] = torch.full_like(found["top_k"], 50)
        found["top_p"] = 0.8 + 0.18 * rand()
    elif keep == "mixed":
        found["temperature"] = torch.where(rand() < 0.1, 0.0 * ones, found["temperature"])
        found["top_k"] = _pick([0, 0, 1, 20, 50, 200], rows, gen).int()
        found["top_p"] = torch.where(rand() < 0.5, 0.8 + 0.18 * rand(), ones)
        found["min_p"] = _pick([0.0, 0.0, 0.05, 0.1], rows, gen).float()
    return found


def _ids(case, gen):
    """Token ids as frequent as words are (the r-th most frequent 1/r as often),
    -1 where a position is padded."""
    rows, vocab = case["rows"], case["vocab"]
    rank = torch.exp(torch.rand((rows,), device="cuda", generator=gen) * math.log(vocab)).long()
    names = torch.randperm(vocab, device="cuda", generator=gen)
    ids = names[(rank - 1).clamp(0, vocab - 1)].int()
    gone = torch.rand((rows,), device="cuda", generator=gen) < case["absent"]
    return torch.where(gone, torch.full_like(ids, -1), ids)


def _normal(rows, width, pad, dtype, gen, scale=1.0):
    out = _padded(rows, width, pad, dtype)
    step = max(1, 2 ** 27 // width)
    for r in range(0, rows, step):
        n = min(step, rows - r)
        out[r:r + n] = (torch.randn((n, width), device="cuda", generator=gen) * scale).to(dtype)
    return out


def _activations(case, gen):
    """Hidden rows of their own size and offset, with a few large columns."""
    rows, width = case["rows"], case["width"]
    x = _normal(rows, width, case["pad"], torch.float32, gen)
    x *= torch.exp(torch.randn((rows, 1), device="cuda", generator=gen))
    x += 0.3 * torch.randn((rows, 1), device="cuda", generator=gen)
    large = torch.randint(width, (4,), device="cuda", generator=gen)
    x[:, large] *= 12.0
    out = _padded(rows, width, case["pad"], DTYPES[case["dtype"]])
    out.copy_(x)
    return out


def prepare(case, seed):
    gen = _generator(seed)
    op, dtype, rows = case["op"], DTYPES[case["dtype"]], case["rows"]
    state = {"case": case}
    if op == "sample":
        state["logits"] = _logits(case, gen)
        state["uniform"] = torch.rand((rows,), device="cuda", generator=gen)
        state.update(_settings(case, gen))
        return state
    width, pad = case["width"], case["pad"]
    if op == "embed":
        state["ids"] = _ids(case, gen)
        state["table"] = _normal(case["vocab"], width, pad, dtype, gen, 0.02)
    elif op == "embed_grad":
        state["ids"] = _ids(case, gen)
        state["grad"] = _normal(rows, width, pad, dtype, gen, 1e-2)
    else:
        state["x"] = _activations(case, gen)
        weight = 1.0 + 0.2 * torch.randn((width,), device="cuda", generator=gen)
        state["weight"] = weight.to(DTYPES[case["weight_dtype"]])
        if op == "norm":
            bias = 0.2 * torch.randn((width,), device="cuda", generator=gen)
            state["bias"] = bias.to(DTYPES[case["weight_dtype"]])
        else:
            state["stats"] = _norm_stats(state["x"])
            state["grad"] = _normal(rows, width, pad, dtype, gen, 1e-2)
    return state


def _norm_stats(x):
    """Mean and 1 / sqrt(variance + eps) of every row, summed in 64 bits."""
    y = x.double()
    mean = y.mean(1)
    return torch.stack([mean, torch.rsqrt(y.var(1, unbiased=False) + EPS)], 1).float()


# ---------------------------------------------------------------------------
# One pass.


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "sample":
        return _plain_sample(state)
    if op == "embed":
        return _plain_embed(state)
    if op == "embed_grad":
        return _plain_embed_grad(state)
    if op == "norm":
        return _plain_norm(state)
    return _plain_norm_grad(state)


def _plain_sample(state):
    """Sums in 64 bits: the draw is a whole number, decided at the border
    between two tokens of a sum over the vocabulary."""
    vocab = state["case"]["vocab"]
    z = state["logits"].float()
    greedy = state["temperature"] == 0
    tau = torch.where(greedy, torch.ones_like(state["temperature"]), state["temperature"])
    k = torch.where(state["top_k"] == 0, torch.full_like(state["top_k"], vocab), state["top_k"])
    k = torch.where(greedy, torch.ones_like(k), k)
    ordered, index = torch.sort(z, dim=1, descending=True, stable=True)
    high = ordered[:, :1].double()
    x = (ordered.double() - high) / tau.double()[:, None]
    w = torch.exp(x)
    keep = torch.arange(vocab, device=z.device) < k[:, None]
    some = torch.where(keep, w, torch.zeros_like(w))
    summed = torch.cumsum(some, 1)
    p = state["top_p"].double()[:, None]
    keep &= (p == 1) | (summed - some < p * summed[:, -1:])
    keep &= x >= torch.log(state["min_p"].double())[:, None]
    mass = torch.zeros_like(w).scatter_(1, index, torch.where(keep, w, torch.zeros_like(w)))
    summed = torch.cumsum(mass, 1)
    whole = summed[:, -1]
    token = (summed <= (state["uniform"].double() * whole)[:, None]).sum(1)
    drawn = (z.gather(1, token[:, None])[:, 0].double() - high[:, 0]) / tau.double()
    return {"token": token.int(), "logprob": (drawn - torch.log(whole)).float()}


def _plain_embed(state):
    ids = state["ids"].long()
    rows = state["table"][ids.clamp(min=0)].float() * state["case"]["scale"]
    return torch.where(ids[:, None] < 0, torch.zeros_like(rows), rows).to(state["table"].dtype)


def _plain_embed_grad(state):
    case = state["case"]
    ids = state["ids"].long()
    total = torch.zeros((case["vocab"] + 1, case["width"]), device=ids.device)
    total.index_add_(0, torch.where(ids < 0, torch.full_like(ids, case["vocab"]), ids),
                     state["grad"].float())
    return (total[:-1] * case["scale"]).to(DTYPES[case["grad_dtype"]])


def _plain_norm(state):
    x = state["x"].float()
    mean = x.mean(1, keepdim=True)
    far = x - mean
    inverse = torch.rsqrt((far * far).mean(1, keepdim=True) + EPS)
    y = far * inverse * state["weight"].float() + state["bias"].float()
    return {"y": y.to(state["x"].dtype), "stats": torch.cat([mean, inverse], 1)}


def _plain_norm_grad(state):
    grad = state["grad"].float()
    inverse = state["stats"][:, 1:]
    unit = (state["x"].float() - state["stats"][:, :1]) * inverse
    d = grad * state["weight"].float()
    dx = inverse * (d - d.mean(1, keepdim=True) - unit * (d * unit).mean(1, keepdim=True))
    kind = state["weight"].dtype
    return {"grad_x": dx.to(state["x"].dtype), "grad_weight": (grad * unit).sum(0).to(kind),
            "grad_bias": grad.sum(0).to(kind)}


def _run_own(state):
    """The framework's call, its configuration, outputs and workspace bound on
    the state's first pass and run on torch's current stream."""
    if "call" not in state:
        state["call"], state["out"] = _bind(state)
    state["call"].run(torch.cuda.current_stream().cuda_stream)
    return state["out"]


def _bind(state):
    from post_processing_amd import logits as lg
    from post_processing_amd import states as st
    from post_processing_amd import ws

    case = state["case"]
    codes = {"f32": ws.DTYPE_F32, "f16": ws.DTYPE_F16, "bf16": ws.DTYPE_BF16}
    op, rows, dtype = case["op"], case["rows"], DTYPES[case["dtype"]]

    def fresh(*size, dtype=torch.float32):
        return torch.empty(size, dtype=dtype, device="cuda")

    if op == "sample":
        shape = lg.make_rows(rows=rows, vocab=case["vocab"], dtype=codes[case["dtype"]],
                             row_stride=case["vocab"] + case["pad"])
        out = {"token": fresh(rows, dtype=torch.int32), "logprob": fresh(rows)}
        call = lg.Sample(shape, state["logits"], state["uniform"], out["token"],
                         logprob=out["logprob"], temperature=state["temperature"],
                         top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"])
        return call, out
    width, stride = case["width"], case["width"] + case["pad"]
    if op == "embed":
        shape = st.make_states(rows=rows, width=width, dtype=codes[case["dtype"]])
        out = fresh(rows, width, dtype=dtype)
        return st.Embed(shape, state["table"], state["ids"], out, vocab=case["vocab"],
                        table_stride=stride, scale=case["scale"]), out
    shape = st.make_states(rows=rows, width=width, dtype=codes[case["dtype"]], row_stride=stride)
    if op == "embed_grad":
        out = fresh(case["vocab"], width, dtype=DTYPES[case["grad_dtype"]])
        return st.EmbedGrad(shape, state["grad"], state["ids"], out, vocab=case["vocab"],
                            grad_dtype=codes[case["grad_dtype"]], scale=case["scale"]), out
    kind = codes[case["weight_dtype"]]
    if op == "norm":
        out = {"y": fresh(rows, width, dtype=dtype), "stats": fresh(rows, 2)}
        return st.LayerNorm(shape, state["x"], out["y"], weight=state["weight"],
                            bias=state["bias"], weight_dtype=kind, eps=EPS,
                            stats=out["stats"]), out
    out = {"grad_x": fresh(rows, width, dtype=dtype),
           "grad_weight": fresh(width, dtype=state["weight"].dtype),
           "grad_bias": fresh(width, dtype=state["weight"].dtype)}
    return st.LayerNormGrad(shape, state["x"], state["stats"], state["grad"],
                            weight=state["weight"], weight_dtype=kind, **out), out


# ---------------------------------------------------------------------------


def work(case):
    """Each input read once and each output written once.  Sampling: difference,
    scale, exponential and sum an element; a gradient row's one product and
    one sum an element; norm's sums and products."""
    op, rows, size = case["op"], case["rows"], SIZES[case["dtype"]]
    if op == "sample":
        return {"bytes": rows * (case["vocab"] * size + 28), "flops": 4 * rows * case["vocab"]}
    cells = rows * case["width"]
    if op == "embed":
        return {"bytes": 2 * cells * size + 4 * rows, "flops": cells}
    if op == "embed_grad":
        out = case["vocab"] * case["width"] * SIZES[case["grad_dtype"]]
        return {"bytes": cells * size + 4 * rows + out, "flops": 2 * cells}
    weights = case["width"] * SIZES[case["weight_dtype"]]
    if op == "norm":
        return {"bytes": 2 * cells * size + 8 * rows + 2 * weights, "flops": 8 * cells}
    return {"bytes": 3 * cells * size + 8 * rows + 3 * weights, "flops": 14 * cells}


def exact(case, seed):
    """The outputs from the definitions in 64 bits."""
    state = prepare(case, seed)
    op = case["op"]
    if op == "sample":
        found = [_exact_draw(state, r) for r in range(case["rows"])]
        return {"token": torch.stack([f[0] for f in found]).int(),
                "logprob": torch.stack([f[1] for f in found])}
    if op == "embed":
        ids = state["ids"].long()
        named = (ids >= 0).double()[:, None] * case["scale"]
        return named * torch.index_select(state["table"], 0, ids.clamp(min=0)).double()
    if op == "embed_grad":
        # Tokens in order, each one's rows one run of a running sum.
        ids, at = torch.sort(state["ids"].long(), stable=True)
        grad = state["grad"].double()[at]
        total = torch.zeros((case["vocab"], case["width"]), dtype=torch.float64, device="cuda")
        names, count = torch.unique_consecutive(ids, return_counts=True)
        ends = torch.cumsum(count, 0)
        for name, n, end in zip(names.tolist(), count.tolist(), ends.tolist()):
            if name >= 0:
                total[name] = grad[end - n:end].sum(0) * case["scale"]
        return total
    x, gamma = state["x"].double(), state["weight"].double()
    if op == "norm":
        mean = x.sum(1) / case["width"]
        variance = (x * x).sum(1) / case["width"] - mean * mean
        inverse = 1.0 / torch.sqrt(variance + EPS)
        y = (x - mean[:, None]) * (inverse[:, None] * gamma) + state["bias"].double()
        return {"y": y, "stats": torch.stack([mean, inverse], 1)}
    # The row's mean and deviation as the forward pass left them.
    mean, inverse = state["stats"].double().unbind(1)
    unit = (x - mean[:, None]) * inverse[:, None]
    grad = state["grad"].double()
    ahead = grad * gamma
    along = (ahead * unit).sum(1, keepdim=True) / case["width"]
    level = ahead.sum(1, keepdim=True) / case["width"]
    return {"grad_x": (ahead - level - along * unit) * inverse[:, None],
            "grad_weight": (grad * unit).sum(0), "grad_bias": grad.sum(0)}


def _exact_draw(state, r):
    """One row's token and log probability: the kept tokens one after the other
    by value, then drawn in vocabulary order."""
    z = state["logits"][r].double()
    tau, k = state["temperature"][r].double(), int(state["top_k"][r])
    p, least = state["top_p"][r].double(), state["min_p"][r].double()
    if tau == 0:
        tau, k = torch.ones_like(tau), 1
    n = min(k or z.numel(), z.numel())
    # Distinct ranks: how many tokens come before, by value and then by index.
    by_value = torch.argsort(-z, stable=True)[:n]
    weight = torch.exp((z[by_value] - z.max()) / tau)
    upto = torch.cumsum(weight, 0)
    if p < 1:
        enough = torch.searchsorted(upto, (p * upto[-1])[None])[0]
        by_value, weight = by_value[:enough + 1], weight[:enough + 1]
    fine = (z[by_value] - z.max()) / tau >= torch.log(least)
    kept, at = torch.sort(by_value[fine])
    upto = torch.cumsum(weight[fine][at], 0)
    place = torch.searchsorted(upto, (state["uniform"][r].double() * upto[-1])[None], right=True)
    return kept[place[0]], torch.log(weight[fine][at][place[0]] / upto[-1])
