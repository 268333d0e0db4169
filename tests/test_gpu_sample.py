"""Tokens drawn from rows of logits against the float64 oracle.

Tokens are equal: weights and sums are FP64 on both sides.  The kernels' weights are
up to 1.6e-13 too small (an exponential of a table and a cubic), so the borders
between tokens, as shares of the whole, are off by less than 2e-13, and a draw differs
only where u lies that near one: a chance of at most V 4e-13 a row, 8e-8 at the 200,003
tokens of the longest drawn ones here (the row of 2^30 has its numbers chosen, and
weights of 1 but for two).  Where a test puts u on a border on purpose, the weights are
equal, and every sum is exact.

The log probability is log(w_t / K): both good to 2e-13, so their ratio's log to 4e-13
and the logarithm's own 2e-16, rounded once to FP32: half a step, E = 2^-24 relative,
and 1e-12.
"""
import numpy as np
import pytest

from oracle import logits as ol
from post_processing_amd import logits as lg
from post_processing_amd import ws

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
TYPES = ["f32", "f16", "bf16"]
CODE = {"f32": ws.DTYPE_F32, "f16": ws.DTYPE_F16, "bf16": ws.DTYPE_BF16}


def _type(dtype):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]


def _dev():
    import torch
    return torch.device("cuda:0")


def _settings(n, **given):
    """One value a row of each setting, None where it is not given."""
    kinds = {"temperature": np.float32, "top_k": np.int32, "top_p": np.float32,
             "min_p": np.float32}
    return {key: None if given.get(key) is None
            else np.broadcast_to(np.asarray(given[key], dtype=kind), (n,)).copy()
            for key, kind in kinds.items()}


def draw(z, u, dtype, pad=0, shift=0, tau=1.0, logprob=True, stream=None, **settings):
    """(exact logits, tokens, log probabilities) of a call."""
    import torch
    rows, V = z.shape
    stride = V + pad
    flat = torch.full((shift + rows * stride + 16,), 3e4, dtype=_type(dtype), device=_dev())
    view = torch.as_strided(flat, (rows, V), (stride, 1), shift)
    view.copy_(torch.from_numpy(np.array(z, order="C")).to(_dev()))
    shape = lg.make_rows(rows=rows, vocab=V, dtype=CODE[dtype], row_stride=stride,
                         temperature=tau)
    on = {k: None if v is None else torch.from_numpy(v).to(_dev()) for k, v in settings.items()}
    token = torch.full((rows,), -77, dtype=torch.int32, device=_dev())
    lp = torch.full((rows,), -77.0, device=_dev()) if logprob else None
    uniform = torch.from_numpy(np.asarray(u, dtype=np.float32)).to(_dev())
    call = lg.Sample(shape, view, uniform, token, logprob=lp, **on)
    torch.cuda.synchronize()
    call.run(stream)
    torch.cuda.synchronize()
    return (view.double().cpu().numpy(), token.cpu().numpy(),
            lp.double().cpu().numpy() if logprob else None)


def check(z, u, dtype, pad=0, shift=0, tau=1.0, **given):
    rows = z.shape[0]
    s = _settings(rows, **given)
    exact, token, lp = draw(z, u, dtype, pad, shift, tau, **s)
    u = np.asarray(u, dtype=np.float32).astype(np.float64)
    for r in range(rows):
        one = lambda key, off: off if s[key] is None else s[key][r].item()  # noqa: E731
        t = one("temperature", float(np.float32(tau)))
        want, wlp = ol.sample(exact[r], u[r], t, one("top_k", 0), one("top_p", 1.0),
                              one("min_p", 0.0))
        assert token[r] == want, (r, token[r], want, u[r], {k: None if v is None else v[r]
                                                             for k, v in s.items()})
        if np.isfinite(wlp):
            assert abs(lp[r] - wlp) <= E * abs(wlp) + 1e-12, (r, lp[r], wlp)
        else:
            assert lp[r] == wlp or (np.isnan(lp[r]) and np.isnan(wlp)), (r, lp[r], wlp)
    return token


def logits(rng, rows, V, scale=None):
    """Rows from peaked to flat."""
    scale = rng.uniform(0.3, 3.0, (rows, 1)) if scale is None else scale
    z = rng.normal(size=(rows, V)) * scale
    hot = rng.integers(0, V, (rows, 6))
    np.put_along_axis(z, hot, rng.uniform(0, 14, (rows, 1)) + rng.normal(size=(rows, 6)), 1)
    return z


MIXES = [dict(), dict(top_k=1), dict(top_k=7), dict(top_k=50), dict(top_p=0.9), dict(top_p=0.3),
         dict(top_p=0.0), dict(min_p=0.05), dict(min_p=1.0), dict(top_k=50, top_p=0.8),
         dict(top_k=40, top_p=0.95, min_p=0.02), dict(top_p=0.99, min_p=0.001),
         dict(top_k=100000000), dict(temperature=0.0)]
SIZES = [1, 2, 7, 8, 9, 63, 64, 65, 255, 1000, 2049, 8192, 8193, 21843, 70001]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", SIZES)
def test_sample_sizes(gpu_lib, dtype, V):
    rng = np.random.default_rng(V)
    n = len(MIXES)
    z = logits(rng, n, V)
    rows = [{**dict(temperature=0.8, top_k=0, top_p=1.0, min_p=0.0), **m} for m in MIXES]
    given = {k: [r[k] for r in rows] for k in rows[0]}
    for _ in range(3):
        check(z, rng.random(n), dtype, **given)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mix", range(len(MIXES)))
@pytest.mark.parametrize("V", [100, 5000, 40001])
def test_sample_settings(gpu_lib, dtype, mix, V):
    """Each combination alone, what it leaves out given as no array."""
    rng = np.random.default_rng(mix)
    check(logits(rng, 24, V), rng.random(24), dtype, tau=0.9, **MIXES[mix])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 5), (0, 1), (24, 8), (7, 3)])
@pytest.mark.parametrize("V", [5, 129, 3001, 33000])
def test_sample_strides_and_starts(gpu_lib, dtype, pad, shift, V):
    rng = np.random.default_rng(V + pad)
    check(logits(rng, 6, V), rng.random(6), dtype, pad, shift, top_k=[0, 3, 20, 0, 0, 1],
          top_p=[1, 1, 0.9, 0.7, 1, 1], min_p=[0, 0, 0, 0, 0.1, 0])


@pytest.mark.parametrize("tau", [1e-3, 0.05, 0.7, 2.0, 30.0, 1e3])
def test_sample_temperatures(gpu_lib, tau):
    rng = np.random.default_rng(5)
    for V in (300, 20011):
        z = logits(rng, 12, V)
        check(z, rng.random(12), "f32", tau=tau)
        check(z, rng.random(12), "bf16", temperature=tau, top_k=30, top_p=0.9)
        check(z, rng.random(12), "f16", temperature=tau, top_p=0.6, min_p=0.01)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("k", [1, 2, 31, 32, 33, 64, 65, 200, 1024, 1025, 5000, 29999, 30000, 30001])
def test_sample_top_k(gpu_lib, dtype, k):
    rng = np.random.default_rng(k)
    z = logits(rng, 10, 30000)
    check(z, rng.random(10), dtype, top_k=k)
    check(z, rng.random(10), dtype, top_k=k, top_p=0.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("p", [1e-6, 0.01, 0.5, 0.9, 0.999, 1 - 2.0 ** -24])
def test_sample_top_p(gpu_lib, dtype, p):
    rng = np.random.default_rng(int(p * 1000))
    for V in (50, 3000, 50001):
        check(logits(rng, 10, V), rng.random(10), dtype, top_p=p)


def test_sample_flat_rows(gpu_lib):
    """All tokens alike: every draw is a border's arithmetic, every cut a tie."""
    rng = np.random.default_rng(8)
    for V in (64, 1000, 4096, 100003):
        z = np.full((9, V), 1.25)
        u = np.concatenate([[0.0, 0.5, 0.25, 1 - 2.0 ** -24], rng.random(5)])
        check(z, u, "bf16")
        check(z, u, "bf16", top_k=[1, 2, 3, V - 1, V, V + 1, 10, 60, 0])
        check(z, u, "f32", top_p=[0.5, 0.25, 0.125, 0.75, 1, 0, 1e-9, 1 - 2.0 ** -24, 0.3])
        check(z, u, "f16", min_p=[1, 0.5, 1, 0.5, 0, 0, 1, 1, 1])


@pytest.mark.parametrize("dtype", TYPES)
def test_sample_ties(gpu_lib, dtype):
    """Few distinct values, so that every cut falls among equal ones, which go by
    index; whole powers of two as weights, so that borders are exact."""
    rng = np.random.default_rng(9)
    for V in (100, 3000, 60001):
        z = rng.integers(-3, 3, (12, V)).astype(float)
        check(z, rng.random(12), dtype, top_k=rng.integers(1, V, 12))
        check(z, rng.random(12), dtype, top_p=rng.random(12))
        check(z, rng.random(12), dtype, top_k=rng.integers(1, V, 12), top_p=rng.random(12))
    z = np.array([[0.0, 0.0, -1.0, -1.0, -np.inf, 0.0]])
    for u in (0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24):
        check(z, [u], dtype, top_k=4)
        check(z, [u], dtype, top_k=3)


def test_sample_zeros_of_either_sign_are_equal(gpu_lib):
    z = np.where(np.arange(50) % 2 == 0, -0.0, 0.0)[None].repeat(4, 0)
    for k in (1, 2, 5):
        got = check(z, [0.0, 0.3, 0.6, 0.99], "f32", top_k=k)
        assert (got < k).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [40, 5000, 40001])
def test_sample_special_rows(gpu_lib, dtype, V):
    low = {"f32": -3.4028234663852886e38, "f16": -65504.0, "bf16": -3.3895313892515355e38}[dtype]
    top = {"f32": 3e38, "f16": 6e4, "bf16": 3e38}[dtype]
    rng = np.random.default_rng(10)
    base = rng.normal(size=V)
    rows = [np.full(V, -np.inf), np.full(V, low), np.full(V, top), base.copy(), base.copy(),
            base.copy(), np.full(V, -np.inf), np.full(V, -np.inf), base * top / 10, base.copy(),
            np.full(V, low), base - 5000.0]
    rows[3][V // 2] = np.nan
    rows[4][V - 1] = np.inf
    rows[5][0] = np.nan
    rows[6][V // 3] = 2.0                              # one token left
    rows[7][[1, V // 2, V - 1]] = [0.0, 1.0, low]      # three, one without weight
    rows[9][rng.random(V) < 0.9] = low
    rows[10][V - 1] = 0.0
    z = np.stack(rows)
    for given in ({}, dict(top_k=5), dict(top_p=0.9), dict(min_p=0.2),
                  dict(top_k=10, top_p=0.7, min_p=0.01), dict(temperature=0.0)):
        for u in (0.0, 0.4, 1 - 2.0 ** -24):
            check(z, np.full(len(z), u), dtype, **given)


def test_sample_settings_outside_their_ranges(gpu_lib):
    z = np.random.default_rng(11).normal(size=(10, 500))
    nan = np.nan
    for given in (dict(temperature=[-1, nan, 1e-4, 2e3, np.inf, 1, 1, 1, 1, 1]),
                  dict(top_k=[-1, -2 ** 31, 3, 0, 1, 2, 3, 4, 5, 6]),
                  dict(top_p=[-0.1, 1.1, nan, np.inf, 0.5, 1, 0, 0.1, 0.2, 0.3]),
                  dict(min_p=[-0.1, 1.1, nan, np.inf, 0.5, 1, 0, 0.1, 0.2, 0.3])):
        check(z, np.full(10, 0.5), "f32", **given)
    check(z, [1.0, -0.1, nan, np.inf, 2.0, 0.0, 0.5, 0.1, 0.9, -np.inf], "bf16")


def test_sample_draws_follow_the_distribution(gpu_lib):
    """Evenly spread numbers draw every token as often as its probability says."""
    rng = np.random.default_rng(12)
    z = rng.normal(size=200) * 2
    n = 4096
    u = (np.arange(n) + 0.5) / n
    _, token, lp = draw(z[None].repeat(n, 0), u, "f32", **_settings(n, top_p=0.95))
    kept, w = ol.kept_tokens(np.float32(z).astype(float), 1.0, 0, float(np.float32(0.95)))
    p = np.zeros(200)
    p[kept] = w / w.sum()
    count = np.bincount(token, minlength=200)
    assert (np.abs(count - n * p) <= 1.0).all()
    np.testing.assert_allclose(lp, np.log(p[token]), rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("rows,V", [(1, 131072), (3, 200003), (64, 32768), (300, 4099), (700, 50001)])
def test_sample_batches(gpu_lib, rows, V):
    """As they come from requests: many rows, each with its own settings."""
    rng = np.random.default_rng(rows)
    for dtype in ("bf16", "f32"):
        check(logits(rng, rows, V), rng.random(rows), dtype,
              temperature=rng.choice([0.0, 0.6, 1.0, 1.3], rows),
              top_k=rng.choice([0, 0, 1, 20, 50, 200], rows),
              top_p=np.where(rng.random(rows) < 0.5, 1.0, rng.uniform(0.5, 0.99, rows)),
              min_p=rng.choice([0, 0, 0.05, 0.1], rows))


@pytest.mark.parametrize("rows,V,dtype", [(257, 131072, "bf16"), (257, 131073, "bf16"), (300, 65537, "f32")])
def test_sample_rows_in_two_turns(gpu_lib, rows, V, dtype):
    """More rows than CUs on both sides of the border between 512 and 1,024 threads a
    row, undecided ones among them."""
    rng = np.random.default_rng(V)
    z = logits(rng, rows, V)
    kinds = np.arange(rows) % 4
    given = dict(temperature=0.9, top_k=np.choose(kinds, [0, 50, 0, 700]),
                 top_p=np.choose(kinds, [1.0, 0.9, 0.8, 0.95]), min_p=np.choose(kinds, [0.0, 0.0, 0.0, 1e-3]))
    check(z, rng.random(rows), dtype, **given)


@pytest.mark.parametrize("rows", [257, 512, 513, 1023, 1024, 1025, 2600])
def test_sample_rows_in_any_order(gpu_lib, rows):
    """More rows than workgroups at work at a time, which take them in an order of
    their own: every row is drawn, with its own settings."""
    rng = np.random.default_rng(rows)
    V = 70001 if rows == 1025 else 9001        # long rows and short ones
    z = logits(rng, rows, V)
    kinds = rng.integers(0, 5, rows)
    given = dict(temperature=np.where(kinds == 0, 0.0, 0.9),
                 top_k=np.choose(kinds, [0, 0, 20, 0, 0]),
                 top_p=np.choose(kinds, [1.0, 0.8, 0.9, 1.0, 1.0]),
                 min_p=np.choose(kinds, [0.0, 0.0, 0.0, 0.05, 0.0]))
    check(z, rng.random(rows), "bf16", **given)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [9001, 60001])
def test_sample_wide_nuclei(gpu_lib, dtype, V):
    """Undecided rows, whose nucleus is thousands of tokens: from a histogram, cut
    in a bin of few logits, of many, and among equal ones."""
    rng = np.random.default_rng(V)
    rows = [rng.normal(size=V) * s for s in (0.01, 0.3, 1.0, 2.0)]
    rows += [np.round(rng.normal(size=V) * 4) / 4, np.round(rng.normal(size=V)),
             np.where(rng.random(V) < 0.3, -np.inf, rng.normal(size=V)),
             rng.normal(size=V) * 1e-4 + 50.0]
    z = np.stack(rows * 3)
    p = np.repeat([0.3, 0.8, 0.995], len(rows))
    check(z, rng.random(len(z)), dtype, top_p=p)
    check(z, rng.random(len(z)), dtype, top_p=p, min_p=np.tile([0.0, 0.2, 0.01, 1e-4], 6))
    check(z, rng.random(len(z)), dtype, top_p=p, top_k=np.tile([600, 2000, 5000, 8000], 6),
          temperature=rng.choice([0.3, 1.0, 20.0], len(z)))


def test_sample_without_logprob_and_without_rows(gpu_lib):
    import torch
    rng = np.random.default_rng(13)
    z = logits(rng, 5, 700)
    u = rng.random(5)
    _, a, _ = draw(z, u, "f32", **_settings(5, top_k=9))
    _, b, _ = draw(z, u, "f32", logprob=False, **_settings(5, top_k=9))
    assert (a == b).all()
    token = torch.full((1,), 5, dtype=torch.int32, device=_dev())
    lg.Sample(lg.make_rows(rows=0, vocab=10), None, None, token).run(None)
    torch.cuda.synchronize()
    assert token.item() == 5


def test_sample_rows_past_32_bits(gpu_lib):
    """Rows that start more than 2^32 elements into their buffer."""
    import torch
    rng = np.random.default_rng(14)
    V, stride, rows = 301, (1 << 30) + 24, 6
    flat = torch.empty((rows - 1) * stride + V, dtype=torch.bfloat16, device=_dev())
    view = torch.as_strided(flat, (rows, V), (stride, 1))
    view.copy_(torch.from_numpy(logits(rng, rows, V)).to(_dev()))
    u = rng.random(rows).astype(np.float32)
    token = torch.empty(rows, dtype=torch.int32, device=_dev())
    call = lg.Sample(lg.make_rows(rows=rows, vocab=V, dtype=ws.DTYPE_BF16, row_stride=stride), view,
                     torch.from_numpy(u).to(_dev()), token)
    call.run(torch.cuda.current_stream().cuda_stream)
    exact = view.double().cpu().numpy()
    want = [ol.sample(exact[r], float(u[r]), 1.0)[0] for r in range(rows)]
    assert token.tolist() == want


def test_sample_longest_row(gpu_lib):
    """2^30 logits: a few above the rest, which together outweigh them or not."""
    import torch
    V = 1 << 30
    z = torch.zeros(1, V, dtype=torch.bfloat16, device=_dev())
    z[0, 12345] = 3.0
    z[0, V - 7] = 2.0
    u = torch.tensor([0.75], device=_dev())
    token = torch.empty(1, dtype=torch.int32, device=_dev())
    lp = torch.empty(1, device=_dev())
    shape = lg.make_rows(rows=1, vocab=V, dtype=ws.DTYPE_BF16)
    lg.Sample(shape, z, u, token, logprob=lp).run(torch.cuda.current_stream().cuda_stream)
    total = V - 2 + np.exp(3.0) + np.exp(2.0)
    want = int(np.floor(0.75 * total - np.exp(3.0) + 1.0))   # one step after 12345
    assert token.item() == want
    assert abs(lp.item() + np.log(total)) < 1e-5
    two = torch.tensor([2], dtype=torch.int32, device=_dev())
    lg.Sample(shape, z, u, token, top_k=two, logprob=lp).run(
        torch.cuda.current_stream().cuda_stream)
    assert token.item() == V - 7
    p = torch.tensor([0.25], device=_dev())
    lg.Sample(shape, z, u, token, top_p=p, logprob=lp).run(torch.cuda.current_stream().cuda_stream)
    # The two, and as many of the first zeros as make up a quarter.
    n = int(np.ceil(0.25 * total - np.exp(3.0) - np.exp(2.0)))
    kept = n + np.exp(3.0) + np.exp(2.0)
    assert token.item() == int(np.floor(0.75 * kept - np.exp(3.0) + 1.0))


def _sets(seed, rows=40, V=30011, dtype="bf16"):
    import torch
    rng = np.random.default_rng(seed)
    z = torch.from_numpy(logits(rng, rows, V)).to(_dev()).to(_type(dtype))
    u = torch.from_numpy(rng.random(rows).astype(np.float32)).to(_dev())
    k = torch.from_numpy(rng.choice([0, 1, 30], rows).astype(np.int32)).to(_dev())
    p = torch.from_numpy(rng.choice([1.0, 0.9], rows).astype(np.float32)).to(_dev())
    token = torch.empty(rows, dtype=torch.int32, device=_dev())
    lp = torch.empty(rows, device=_dev())
    shape = lg.make_rows(rows=rows, vocab=V, dtype=CODE[dtype], temperature=0.8)
    return lg.Sample(shape, z, u, token, top_k=k, top_p=p, logprob=lp), (z, u, token, lp)


@pytest.mark.parametrize("rows,V", [(1, 131072), (40, 30011), (300, 5000)])
def test_sample_two_streams_at_once(gpu_lib, rows, V):
    import torch
    sets = [_sets(s, rows, V) for s in (1, 2)]
    want = []
    for call, (_, _, token, lp) in sets:
        call.run(torch.cuda.current_stream().cuda_stream)
        want.append((token.clone(), lp.clone()))
        token.fill_(-7)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for (call, _), s in zip(sets, streams):
            call.run(s.cuda_stream)
    torch.cuda.synchronize()
    for (_, (_, _, token, lp)), (a, b) in zip(sets, want):
        assert torch.equal(token, a) and torch.equal(lp, b)


@pytest.mark.parametrize("rows,V", [(1, 131072), (40, 30011), (300, 5000)])
def test_sample_captured_and_replayed(gpu_lib, rows, V):
    import torch
    call, (z, u, token, lp) = _sets(3, rows, V)
    twin, (z2, u2, token2, lp2) = _sets(3, rows, V)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call.run(torch.cuda.current_stream().cuda_stream)
    for i in range(4):
        gen = torch.Generator(device="cuda").manual_seed(20 + i)
        z.copy_(torch.randn(z.shape, device=_dev(), generator=gen) * (1 + i))
        u.copy_(torch.rand(u.shape, device=_dev(), generator=gen))
        z2.copy_(z)
        u2.copy_(u)
        token.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        twin.run(torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(token, token2) and torch.equal(lp, lp2), i
