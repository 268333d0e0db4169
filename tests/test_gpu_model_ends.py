"""The operators at a language model's two ends run together, as a model runs
them: tokens are looked up, normalised, answered with logits and drawn; a loss's
gradient goes back the same way.

Each stage is held to the float64 oracle on the inputs it was given, with the
tolerances its own tests derive.  The whole gradient is held to differences of a
float64 forward pass: every stage is a sum of fewer than 700 terms, so off by
less than 700 E = 4.2e-5 of its terms' sizes, five stages by 2.1e-4; the sizes are
those of the sum over all weights.
"""
import numpy as np
import pytest

import test_gpu_logits as tl
import test_gpu_sample as ts
import test_gpu_states as tst
from oracle import logits as ol
from oracle import states as os_
from post_processing_amd import logits as lg
from post_processing_amd import states as st
from post_processing_amd import ws

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def _dev():
    import torch
    return torch.device("cuda:0")


def _tensor(x, dtype=None):
    import torch
    return torch.from_numpy(np.asarray(x)).to(_dev()).to(dtype or torch.float32)


def _np(x):
    return x.double().cpu().numpy()


def test_a_training_step(gpu_lib):
    import torch
    rng = np.random.default_rng(0)
    rows, width, vocab, eps, scale = 96, 65, 501, 1e-5, 8.0
    ids = rng.integers(0, vocab, rows)
    ids[5:9] = -1
    targets = np.where(ids < 0, -1, rng.integers(0, vocab, rows))
    table, head = rng.normal(size=(vocab, width)) * 0.1, rng.normal(size=(vocab, width)) * 0.3
    weight, bias = 1 + 0.2 * rng.normal(size=width), 0.1 * rng.normal(size=width)
    T, H, W, B = (_tensor(x) for x in (table, head, weight, bias))
    i, t = _tensor(ids, torch.int32), _tensor(targets, torch.int32)
    new = lambda *s: torch.empty(s, device=_dev())  # noqa: E731
    x, y, stats = new(rows, width), new(rows, width), new(rows, 2)
    shape = st.make_states(rows=rows, width=width)
    stream = torch.cuda.current_stream().cuda_stream
    st.Embed(shape, T, i, x, vocab=vocab, scale=scale).run(stream)
    st.LayerNorm(shape, x, y, weight=W, bias=B, eps=eps, stats=stats).run(stream)
    z = y @ H.t()
    lrows = lg.make_rows(rows=rows, vocab=vocab)
    logprob, lstats = new(rows), new(rows, 2)
    lg.LogProbs(lrows, z, targets=t, logprob=logprob, stats=lstats).run(stream)
    up = torch.full((rows,), -1.0 / rows, device=_dev())
    dz = torch.empty_like(z)
    lg.LogProbsGrad(lrows, z, lstats, dz, targets=t, grad_logprob=up).run(stream)
    dy = dz @ H
    dx, dw, db, dt = new(rows, width), new(width), new(width), new(vocab, width)
    st.LayerNormGrad(shape, x, stats, dy, weight=W, grad_x=dx, grad_weight=dw,
                     grad_bias=db).run(stream)
    st.EmbedGrad(shape, dx, i, dt, vocab=vocab, scale=scale).run(stream)
    torch.cuda.synchronize()

    # Stage by stage, on the inputs each was given.
    want = os_.embed(_np(T), ids, scale)
    tst.assert_close(_np(x), want, 2 * E * np.abs(want), "embed")
    _, _, tol = tst.norm_tolerances(_np(x), _np(W), _np(B), float(np.float32(eps)), "f32")
    tst.assert_close(_np(y), os_.layernorm(_np(x), _np(W), _np(B), float(np.float32(eps))), tol, "y")
    for r in range(rows):
        lp = ol.log_softmax(_np(z[r]), 1.0)
        m, logsum = ol.stats(_np(z[r]), 1.0)
        at = max(int(targets[r]), 0)
        w = ol.token_logprob(lp, int(targets[r]))
        tl.assert_close(_np(logprob[r]), w,
                        tl.logprob_tol(_np(z[r])[at], m, 1.0, logsum, w, vocab), f"row {r}")
    sums = os_.embed_grad(_np(dx), ids, vocab, scale)
    size = os_.embed_grad(np.abs(_np(dx)), ids, vocab, scale)
    tst.assert_close(_np(dt), sums, (rows + 3) * E * size, "grad_table")

    # All of it against differences of the loss in float64.
    def loss(table, weight, bias):
        y = os_.layernorm(os_.embed(table, ids, scale), weight, bias, eps)
        z = y @ head.T
        z -= z.max(1, keepdims=True)
        lp = z - np.log(np.exp(z).sum(1, keepdims=True))
        return -np.where(targets >= 0, lp[np.arange(rows), np.maximum(targets, 0)], 0.0).sum() / rows

    for _ in range(4):
        d = [rng.normal(size=s) for s in (table.shape, (width,), (width,))]
        h = 1e-5
        ahead = loss(table + h * d[0], weight + h * d[1], bias + h * d[2])
        back = loss(table - h * d[0], weight - h * d[1], bias - h * d[2])
        terms = [a * b for a, b in zip(d, (_np(dt), _np(dw), _np(db)))]
        along = sum(x.sum() for x in terms)
        whole = sum(np.abs(x).sum() for x in terms)
        # (a difference in float64: 1e-16 / h of the loss, and h^2)
        assert abs((ahead - back) / (2 * h) - along) <= 2.1e-4 * whole + 1e-8


def _bigrams(seed, streams, vocab, steps, dtype):
    """A model whose answer to a token is a row of a table, normalised: lookup,
    norm and draw, `steps` times over."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind = ts._type(dtype)
    table = (torch.randn(vocab, vocab, device=_dev(), generator=gen)).to(kind)
    weight = (3 + torch.rand(vocab, device=_dev(), generator=gen)).to(kind)
    ids = torch.randint(vocab, (streams,), device=_dev(), generator=gen, dtype=torch.int32)
    shape = st.make_states(rows=streams, width=vocab, dtype=ts.CODE[dtype])
    rows = lg.make_rows(rows=streams, vocab=vocab, dtype=ts.CODE[dtype])
    settings = {"temperature": torch.rand(streams, device=_dev(), generator=gen) + 0.3,
                "top_k": torch.randint(0, 40, (streams,), device=_dev(), generator=gen,
                                       dtype=torch.int32),
                "top_p": 0.5 + 0.5 * torch.rand(streams, device=_dev(), generator=gen)}
    calls, kept = [], []
    token = ids
    for _ in range(steps):
        x = torch.empty(streams, vocab, device=_dev(), dtype=kind)
        z = torch.empty_like(x)
        u = torch.rand(streams, device=_dev(), generator=gen)
        new = torch.empty(streams, device=_dev(), dtype=torch.int32)
        calls += [st.Embed(shape, table, token, x, vocab=vocab),
                  st.LayerNorm(shape, x, z, weight=weight),
                  lg.Sample(rows, z, u, new, **settings)]
        kept.append((token, x, z, u, new))
        token = new
    return calls, kept, table, weight, settings


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("streams,vocab", [(7, 333), (40, 2100)])
def test_generation(gpu_lib, dtype, streams, vocab):
    import torch
    calls, kept, table, weight, settings = _bigrams(1, streams, vocab, 4, dtype)
    stream = torch.cuda.current_stream().cuda_stream
    for c in calls:
        c.run(stream)
    torch.cuda.synchronize()
    s = {k: v.cpu().numpy() for k, v in settings.items()}
    for token, x, z, u, new in kept:
        ids = token.cpu().numpy()
        assert np.array_equal(_np(x), os_.embed(_np(table), ids, 1.0))
        _, _, tol = tst.norm_tolerances(_np(x), _np(weight), None, float(np.float32(1e-5)), dtype)
        tst.assert_close(_np(z), os_.layernorm(_np(x), _np(weight), None, float(np.float32(1e-5))),
                         tol, "norm")
        for r in range(streams):
            want, _ = ol.sample(_np(z[r]), float(u[r]), float(s["temperature"][r]),
                                int(s["top_k"][r]), float(s["top_p"][r]))
            assert int(new[r]) == want, r


def test_generation_captured(gpu_lib):
    """The loop as one graph, replayed on new tables and numbers."""
    import torch
    calls, kept, table, weight, _ = _bigrams(2, 9, 700, 5, "bf16")
    twin, kept2, table2, _, _ = _bigrams(2, 9, 700, 5, "bf16")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in calls:
            c.run(torch.cuda.current_stream().cuda_stream)
    for i in range(4):
        gen = torch.Generator(device="cuda").manual_seed(50 + i)
        table.copy_(torch.randn(table.shape, device=_dev(), generator=gen))
        table2.copy_(table)
        for a, b in zip(kept, kept2):
            a[3].copy_(torch.rand(9, device=_dev(), generator=gen))
            b[3].copy_(a[3])
            a[4].fill_(-5)
        graph.replay()
        torch.cuda.synchronize()
        for c in twin:
            c.run(torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        for a, b in zip(kept, kept2):
            assert torch.equal(a[4], b[4]) and torch.equal(a[2], b[2]), i
