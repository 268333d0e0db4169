"""The operators over rows of logits against the float64 oracle.

Tolerances, with E = 2^-24 the half step of FP32 (relative):

* an exponential's argument t = (z - max) log2(e) / tau carries three
  roundings, so 3 E |t| absolute; 2^t adds at most 2 E relative.  Summed with
  weights 2^t the first is at most 3 E x max_x(x 2^-x) < 2 E; the sum itself
  adds at most one E per addition on any element's way, at most ceil(V / 64)
  additions in a lane and 64 to join lanes, waves and workgroups:
      dS / S <= (ceil(V / 64) + 64) E + 4 E          =: SUM(V)
* log S: SUM(V) absolute and 4 E |log S| for the function and its rounding;
* x - max / tau: 3 E relative; the final subtraction E of the result;
* entropy log S - U / S: U's terms e d have 3 E |t| more than e's, weighted
  with x^2 2^-x < 2, so U / S is off by SUM(V) |U / S| + 2 SUM(V) + 8 E (1 +
  |U / S|) in all;
* a gradient's p = 2^(t - log2 S): the argument's error is 4 E (|t| + |log2 S|)
  absolute, p's that times log 2 and 3 E and the statistic's SUM(V) relative;
  the exponential instruction returns 0 for results below FP32's smallest
  normal, so p is off by up to 2^-126 besides, whatever its own size.
  Each product and sum of the formula adds E of its terms' magnitudes (fewer
  than 8 of them), and the result is rounded to the logits' type: half a step
  (and half the smallest step of FP16).
"""
import math

import numpy as np
import pytest

from oracle import logits as ol
from post_processing_amd import logits as lg
from post_processing_amd import ws

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
CODE = {"f32": ws.DTYPE_F32, "f16": ws.DTYPE_F16, "bf16": ws.DTYPE_BF16}
SMALLEST = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def _torch_type(dtype):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]


def _dev():
    import torch
    return torch.device("cuda:0")


def _sum_tol(V):
    return (math.ceil(V / 64) + 68) * E


class Matrix:
    """Rows of logits on the GPU at a chosen offset and stride inside a larger
    buffer of a marker value, and their exact values in float64."""

    def __init__(self, z, dtype, pad=0, shift=0, marker=7.0):
        import torch
        rows, V = z.shape
        self.stride = V + pad
        self.marker = marker
        self.flat = torch.full((shift + rows * self.stride + 16,), marker,
                               dtype=_torch_type(dtype), device=_dev())
        self.shift = shift
        self.shape = (rows, V)
        self.dtype = dtype
        self.view = torch.as_strided(self.flat, (rows, V), (self.stride, 1), shift)
        if z.size:
            self.view.copy_(torch.from_numpy(np.array(z, order="C")).to(_dev()))
        self.z = self.view.double().cpu().numpy()

    def rows(self, tau=1.0):
        return lg.make_rows(rows=self.shape[0], vocab=self.shape[1], dtype=CODE[self.dtype],
                            row_stride=self.stride, temperature=tau)

    def outside_untouched(self):
        flat = self.flat.clone()
        import torch
        torch.as_strided(flat, self.shape, (self.stride, 1), self.shift).fill_(self.marker)
        return bool((flat == self.marker).all())


def _logits(rng, rows, V, scale=3.0):
    z = rng.normal(size=(rows, V)) * scale
    if V > 8:
        z[np.arange(rows), rng.integers(0, V, rows)] += 6.0
    return z


def _tau32(tau):
    return float(np.float32(tau))


def run_logprobs(mat, tau=1.0, targets=None, k=0, entropy=True, stats=True, stream=None):
    import torch
    rows = mat.shape[0]
    d = _dev()
    f = lambda *s: torch.full(s, -12345.0, dtype=torch.float32, device=d)  # noqa: E731
    out = {"entropy": f(rows) if entropy else None, "stats": f(rows, 2) if stats else None,
           "top": torch.full((rows, k, 2), -99, dtype=torch.int32, device=d) if k else None,
           "logprob": f(rows) if targets is not None else None}
    t = torch.from_numpy(np.asarray(targets, dtype=np.int32)).to(d) if targets is not None else None
    call = lg.LogProbs(mat.rows(tau), mat.view, targets=t, logprob=out["logprob"],
                       entropy=out["entropy"], top_k=k, top=out["top"], stats=out["stats"])
    torch.cuda.synchronize()
    call.run(stream)
    torch.cuda.synchronize()
    got = {key: v.cpu().numpy() for key, v in out.items() if v is not None}
    if k:
        got["top_id"] = got["top"][:, :, 1]
        got["top_score"] = np.ascontiguousarray(got["top"][:, :, 0]).view(np.float32)
    got["device"] = out
    return got


def logprob_tol(z, m, tau, logsum, value, V):
    d = np.abs((z - m) / tau)
    return 3 * E * d + _sum_tol(V) + 4 * E * abs(logsum) + 2 * E * np.abs(value) + 1e-37


def assert_close(got, want, tol, what=""):
    got, want, tol = np.broadcast_arrays(np.asarray(got, dtype=np.float64), want, tol)
    with np.errstate(over="ignore"):          # what FP32 cannot hold is an infinity in it
        want = np.where(np.isinf(want.astype(np.float32)), want.astype(np.float32), want)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    fine = np.isfinite(want) & np.isfinite(got)
    assert (same | fine).all(), f"{what}: non-finite values differ"
    err = np.where(same | ~fine, 0.0, np.abs(np.where(fine, got, 0) - np.where(fine, want, 0)))
    worst = err - np.where(same, np.inf, tol)
    at = np.unravel_index(np.argmax(worst), worst.shape)
    assert (worst <= 0).all(), f"{what}: error {err[at]:.3e} over {tol[at]:.3e} at {at}"


def check_logprobs(mat, tau=1.0, targets=None, k=0, entropy=True, stats=True, got=None):
    got = got or run_logprobs(mat, tau, targets, k, entropy, stats)
    tau = _tau32(tau)
    V = mat.shape[1]
    for r in range(mat.shape[0]):
        z = mat.z[r]
        lp = ol.log_softmax(z, tau)
        m, logsum = ol.stats(z, tau)
        plain = np.isfinite(logsum)
        ls = logsum if plain else 0.0
        m0 = m if np.isfinite(m) else 0.0
        if targets is not None:
            t = int(targets[r])
            want = ol.token_logprob(lp, t)
            zt = z[t] if 0 <= t < V and np.isfinite(z[t]) else m0
            w = want if np.isfinite(want) else 0.0
            assert_close(got["logprob"][r], want, logprob_tol(zt, m0, tau, ls, w, V), f"row {r}")
        if entropy:
            h = ol.entropy(lp)
            ratio = abs(ls - h) if np.isfinite(h) else 0.0
            tol = (_sum_tol(V) * (3 + ratio) + 8 * E * (1 + ratio) + 4 * E * abs(ls)
                   + 2 * E * abs(h if np.isfinite(h) else 0.0))
            assert_close(got["entropy"][r], h, tol, f"entropy of row {r}")
        if stats:
            if np.isnan(lp).any():
                assert np.isnan(got["stats"][r, 1])
            else:
                assert got["stats"][r, 0] == np.float32(m)
                assert_close(got["stats"][r, 1], logsum, _sum_tol(V) + 4 * E * abs(ls),
                             f"logsum of row {r}")
        if k:
            ids = ol.best(z, k)
            np.testing.assert_array_equal(got["top_id"][r], ids, err_msg=f"row {r}")
            want = lp[ids]
            zi = np.where(np.isfinite(z[ids]), z[ids], m0)
            assert_close(got["top_score"][r], want,
                         logprob_tol(zi, m0, tau, ls, np.where(np.isfinite(want), want, 0), V),
                         f"scores of row {r}")
    return got


SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (1, 9), (4, 63), (3, 64), (2, 65), (7, 255), (2, 1000),
         (3, 2049), (2, 4097), (1, 8192), (2, 21843), (1, 70001)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V", SIZES)
def test_logprobs_sizes(gpu_lib, dtype, rows, V):
    rng = np.random.default_rng(rows * 100003 + V)
    mat = Matrix(_logits(rng, rows, V), dtype)
    targets = rng.integers(0, V, rows)
    check_logprobs(mat, 1.0, targets, k=min(V, 20))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 5), (0, 1), (24, 8), (7, 3)])
@pytest.mark.parametrize("V", [5, 129, 3001])
def test_logprobs_strides_and_starts(gpu_lib, dtype, pad, shift, V):
    rng = np.random.default_rng(V + pad)
    mat = Matrix(_logits(rng, 5, V), dtype, pad, shift, marker=1e4)   # padding would win
    check_logprobs(mat, 0.7, rng.integers(0, V, 5), k=min(V, 32))
    assert mat.outside_untouched()


@pytest.mark.parametrize("k", [0, 1, 2, 5, 31, 32])
@pytest.mark.parametrize("V", [32, 100, 5000, 40000])
def test_logprobs_k(gpu_lib, k, V):
    rng = np.random.default_rng(k)
    mat = Matrix(_logits(rng, 4, V), "bf16")
    check_logprobs(mat, 1.3, rng.integers(0, V, 4), k=k, entropy=(k % 2 == 0), stats=False)


@pytest.mark.parametrize("tau", [1e-3, 0.1, 1.0, 3.0, 1e3])
def test_logprobs_temperatures(gpu_lib, tau):
    rng = np.random.default_rng(5)
    mat = Matrix(_logits(rng, 6, 777), "f32")
    check_logprobs(mat, tau, rng.integers(0, 777, 6), k=8)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tau", [1e-3, 1.0, 1e3])
def test_logprobs_huge_logits(gpu_lib, dtype, tau):
    """Logits of every magnitude up to the type's largest, of either sign, alone
    and with equals of the maximum: exponents whose parts would overflow."""
    rng = np.random.default_rng(23)
    top = {"f32": 3.0e38, "bf16": 3.0e38, "f16": 6.0e4}[dtype]
    rows = []
    for scale in [1e3, 1e5, 1.5e8, 2e8, 4e8, 1e12, 1e30, 1e38]:
        scale = min(scale, top / 3)
        z = rng.uniform(0.5, 1.0, 600) * scale
        rows += [z, -z, np.concatenate([z[:300], -z[300:]]),
                 np.where(np.arange(600) % 50 == 7, z.max(), rng.normal(size=600)),
                 np.full(600, -scale), z.max() + rng.normal(size=600)]
    z = np.stack(rows)
    check_logprobs(Matrix(z, dtype), tau, rng.integers(0, 600, len(z)), k=8)
    check_logprobs(Matrix(np.tile(z, (1, 20)), dtype), tau, rng.integers(0, 600, len(z)), k=8)


@pytest.mark.parametrize("mode", [0, 1])
def test_distill_huge_logits(gpu_lib, mode):
    rng = np.random.default_rng(24)
    for dtype, scale in [("bf16", 2e8), ("bf16", 1e30), ("f16", 5e4), ("f32", 1e12)]:
        z = np.stack([rng.normal(size=900) * 10 + scale, rng.uniform(-1, 1, 900) * scale,
                      np.full(900, -scale), rng.normal(size=900)])
        mat = Matrix(z, dtype)
        ids, scores = make_teacher(rng, mat.z, 12, mode)
        ids[0, 0] = int(np.argmax(mat.z[0]))
        ids[0, 1:] = np.where(ids[0, 1:] == ids[0, 0], -1, ids[0, 1:])
        check_distill(mat, 1.0, ids, scores, mode, np.ones(4))
        check_distill(mat, 1.0, ids, scores, mode, np.ones(4), separate=True)


def special_rows(V, dtype):
    """Rows where a mask, a value or a tie makes the arithmetic go wrong."""
    rng = np.random.default_rng(17)
    low = {"f32": -3.4028234663852886e38, "f16": -65504.0, "bf16": -3.3895313892515355e38}[dtype]
    rows = [np.full(V, -np.inf), np.full(V, low), np.zeros(V), np.full(V, -7.25)]
    one = np.full(V, -np.inf)
    one[V // 2] = 1.5
    rows.append(one)
    few = np.full(V, -np.inf)
    few[rng.choice(V, min(V, 5), replace=False)] = rng.normal(size=min(V, 5))
    rows.append(few)
    masked = rng.normal(size=V)
    masked[rng.random(V) < 0.9] = low
    rows.append(masked)
    last = np.full(V, low)
    last[-1] = 3.0
    rows.append(last)
    ties = rng.integers(0, 3, V).astype(np.float64)
    rows.append(ties)
    zeros = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    rows.append(zeros)
    nan = rng.normal(size=V)
    nan[V // 3] = np.nan
    rows.append(nan)
    pinf = rng.normal(size=V)
    pinf[V // 4] = np.inf
    rows.append(pinf)
    rows.append(np.full(V, np.nan))
    climb = np.linspace(-40.0, 40.0, V)
    rows.append(climb)
    rows.append(climb[::-1])
    big = rng.normal(size=V) * 1e4
    rows.append(big)
    return np.stack(rows)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 6, 64, 300, 2500, 9001, 33000])
def test_logprobs_special_rows(gpu_lib, dtype, V):
    z = special_rows(V, dtype)
    mat = Matrix(z, dtype)
    rng = np.random.default_rng(V)
    targets = rng.integers(0, V, len(z))
    targets[4] = V // 2
    check_logprobs(mat, 1.0, targets, k=min(V, 32))
    check_logprobs(mat, 0.5, targets, k=min(V, 3))


@pytest.mark.parametrize("V", [70, 20000])
def test_logprobs_ties_across_the_whole_row(gpu_lib, V):
    """Few distinct values, a constant row and a step: the lowest indices of
    the tied value, wherever they lie."""
    rng = np.random.default_rng(9)
    z = np.stack([np.where(np.arange(V) > V - 12, 1.0, 0.0),
                  np.where(np.arange(V) % 97 == 3, 2.0, 1.0),
                  rng.integers(0, 2, V).astype(np.float64),
                  np.where(np.arange(V) == V - 1, 5.0, -np.inf)])
    for dtype in ("bf16", "f32"):
        for k in (1, 20, 32):
            check_logprobs(Matrix(z, dtype), 1.0, None, k=k)


def test_logprobs_signalling_nan(gpu_lib):
    """A NaN of any pattern counts as -inf in the order of the alternatives."""
    import torch
    mat = Matrix(_logits(np.random.default_rng(3), 2, 500), "bf16")
    bits = mat.view.view(torch.int16)
    bits[0, 10] = 0x7f81                    # a signalling pattern
    bits[1, 499] = -0x7f                    # 0xff81
    mat.z = mat.view.double().cpu().numpy()
    mat.z[0, 10] = np.nan
    mat.z[1, 499] = np.nan
    check_logprobs(mat, 1.0, [3, 4], k=32)


def test_logprobs_targets_outside(gpu_lib):
    mat = Matrix(_logits(np.random.default_rng(1), 5, 50), "f32")
    check_logprobs(mat, 1.0, [-1, 50, -2, 49, 2 ** 31 - 1], k=2)


def test_logprobs_same_bits_each_time(gpu_lib):
    mat = Matrix(_logits(np.random.default_rng(2), 9, 50001), "bf16")
    a = run_logprobs(mat, 1.0, np.arange(9), k=20)
    b = run_logprobs(mat, 1.0, np.arange(9), k=20)
    for key in ("logprob", "entropy", "stats", "top"):
        np.testing.assert_array_equal(a[key].view(np.int32), b[key].view(np.int32))


def test_logprobs_many_short_rows(gpu_lib):
    rng = np.random.default_rng(4)
    mat = Matrix(_logits(rng, 3001, 37), "f16")
    check_logprobs(mat, 1.0, rng.integers(0, 37, 3001), k=4)


def _repeated(rows, z):
    """`rows` rows that repeat z's, so the later ones can be held to the first
    bit for bit."""
    return np.broadcast_to(z[np.arange(rows) % len(z)], (rows, z.shape[1]))


@pytest.mark.parametrize("dtype,V,pad,shift", [("f32", 50003, 0, 0), ("bf16", 99001, 3, 1),
                                               ("f16", 131072, 0, 0)])
def test_logprobs_many_long_rows(gpu_lib, dtype, V, pad, shift):
    """Rows too many to split, long enough for the widest workgroups: masked,
    tied, NaN and ordinary ones, each several times over."""
    z = special_rows(V, dtype)
    mat = Matrix(_repeated(300, z), dtype, pad, shift, marker=1e4)
    n = len(z)
    targets = (np.arange(300) % n) * 1009 % V
    got = run_logprobs(mat, 1.0, targets, k=32)
    first = Matrix(z, dtype)
    first.z = mat.z[:n]
    check_logprobs(first, 1.0, targets[:n], k=32, got={key: got[key][:n] for key in got
                                                       if key != "device"})
    for key in ("logprob", "entropy", "stats", "top"):
        np.testing.assert_array_equal(got[key].view(np.int32),
                                      got[key][np.arange(300) % n].view(np.int32))
    assert mat.outside_untouched()


@pytest.mark.parametrize("V", [1 << 20, (1 << 20) + 5])
def test_logprobs_very_long_row(gpu_lib, V):
    rng = np.random.default_rng(V)
    z = np.concatenate([_logits(rng, 2, V), special_rows(V, "bf16")[[4, 5, 8, 10, 13]]])
    check_logprobs(Matrix(z, "bf16", 1, 1), 1.0, rng.integers(0, V, 7), k=32)


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("dtype,rows,V", [("f32", 3, 300001), ("f32", 300, 140001),
                                          ("bf16", 2, 700001), ("bf16", 300, 99001)])
def test_distill_long_rows(gpu_lib, mode, dtype, rows, V):
    """Rows past what a workgroup holds, few and many, where the listed tokens'
    marks limit a part."""
    rng = np.random.default_rng(V)
    z = _logits(rng, 2, V)
    mat = Matrix(_repeated(rows, z), dtype, 1, 1)
    ids, scores = make_teacher(rng, mat.z[:2], 70, mode)
    ids[0, 3], ids[1, 5] = V - 1, 0
    at = np.arange(rows) % 2
    g = np.ones(rows)
    loss, grad, _, _ = run_distill(mat, 1.0, ids[at], scores[at], mode, g)
    # The same row at a start that lies alike within 16 bytes: the same bits.
    vec = 4 if dtype == "f32" else 8
    first = {}
    for r in range(rows):
        f = first.setdefault((r % 2, (1 + r * mat.stride) % vec), r)
        assert loss[r] == loss[f] and (grad[r] == grad[f]).all()
    small = Matrix(z, dtype, 1, 1)
    check_distill(small, 1.0, ids, scores, mode, g[:2])
    check_distill(small, 1.0, ids, scores, mode, g[:2], separate=True)
    want, _, _ = ol.distill(mat.z[0], 1.0, scores[0].astype(np.float64), ids[0], mode)
    assert abs(loss[0] - want) <= 4 * (_sum_tol(V) + 16 * E) * 20


@pytest.mark.parametrize("dtype,rows,V,pad", [("bf16", 1100, 65537, 3), ("f32", 700, 50001, 0),
                                              ("f16", 20000, 3501, 11), ("bf16", 300, 262144, 0),
                                              ("bf16", 9000, 8192, 0)])
def test_matrices_past_the_caches(gpu_lib, dtype, rows, V, pad):
    """Every operator on matrices of more than 128 MiB: the first rows against
    the oracle, the others, which repeat them, against those."""
    rng = np.random.default_rng(rows)
    few, k = 4, 20
    z = _logits(rng, few, V)
    z[2, rng.random(V) < 0.97] = -np.inf
    mat = Matrix(_repeated(rows, z), dtype, pad)
    first = Matrix(z, dtype, pad)
    mat.z = first.z
    at = np.arange(rows) % few
    targets = np.array([3, V - 1, int(np.argmax(z[2])), 0])
    got = run_logprobs(mat, 0.9, targets[at], k=k)
    head = {key: got[key][:few] for key in got if key != "device"}
    check_logprobs(first, 0.9, targets, k=k, got=head)
    vec = 4 if dtype == "f32" else 8
    same = {}
    lead = np.array([same.setdefault((r % few, r * mat.stride % vec), r) for r in range(rows)])
    for key in ("logprob", "entropy", "stats", "top"):
        np.testing.assert_array_equal(got[key].view(np.int32), got[key][lead].view(np.int32))
    ids, scores = make_teacher(rng, first.z, k, ol.TAIL)
    g = np.ones(rows)
    loss, grad, _, _ = run_distill(mat, 0.9, ids[at], scores[at], ol.TAIL, g)
    lsep, gsep, _, _ = run_distill(mat, 0.9, ids[at], scores[at], ol.TAIL, g, separate=True)
    check_distill(first, 0.9, ids, scores, ol.TAIL, g[:few])
    small, sgrad, _, _ = run_distill(first, 0.9, ids, scores, ol.TAIL, g[:few])
    for l, d in ((loss, grad), (lsep, gsep)):
        np.testing.assert_allclose(l[:few], small, rtol=1e-5, atol=40 * _sum_tol(V))
        for r in range(few):
            np.testing.assert_allclose(d[r], sgrad[r], rtol=2.1 * HALF[dtype] + 4 * _sum_tol(V),
                                       atol=8 * _sum_tol(V) + 2 * SMALLEST[dtype])
        assert (l == l[lead]).all()
        assert all(np.array_equal(d[r], d[lead[r]]) for r in range(0, rows, 7))
    del grad, gsep, lsep
    st = row_stats(first, 0.9)[at]
    ent = np.array([ol.entropy(ol.log_softmax(r, _tau32(0.9))) for r in first.z])[at]
    up = rng.normal(size=few)[at]
    check_logprobs_grad(first, 0.9, targets, up[:few], up[:few])
    want = run_logprobs_grad(first, 0.9, st[:few], targets, up[:few], ent[:few], up[:few])
    whole = run_logprobs_grad(mat, 0.9, st, targets[at], up, ent, up, in_place=True)
    for r in (0, 1, 2, 3, rows // 2, rows - 1):
        np.testing.assert_allclose(whole[r], want[r % few], rtol=2.1 * HALF[dtype],
                                   atol=1e-6 + 2 * SMALLEST[dtype])


def test_distill_row_of_more_parts_than_lanes(gpu_lib):
    """A row so long that the marks' limit gives more than 64 parts; logits
    spread so that every part's sum matters."""
    V = 20_000_003
    rng = np.random.default_rng(3)
    mat = Matrix(rng.normal(size=(1, V)), "f16")
    ids = np.array([[5, V - 1, V // 2]])
    scores = np.log(np.array([[0.2, 0.3, 0.1]]))
    z = mat.z[0]
    e = np.exp(z - z.max())
    lse = z.max() + np.log(e.sum())
    rest = e.sum() - e[ids[0]].sum()
    tail = z.max() + np.log(rest) - lse
    s32 = scores.astype(np.float32).astype(np.float64)[0]
    q = np.exp(s32)
    want = (q * (s32 - (z[ids[0]] - lse))).sum() + (1 - q.sum()) * (np.log(1 - q.sum()) - tail)
    loss, grad, stats, got_tail = run_distill(mat, 1.0, ids, scores, ol.TAIL, np.full(1, 1e6),
                                              separate=True)
    # A lane adds at most V / (64 parts of 256 lanes) terms before it joins.
    tol = (V / (64 * 256) + 200) * E
    assert abs(loss[0] - want) <= 4 * tol and abs(float(got_tail[0]) - tail) <= 4 * tol + 2 * E
    p = np.exp(z - lse)
    dz = 1e6 * np.where(np.isin(np.arange(V), ids[0]), p, p * (1 - (1 - q.sum()) / np.exp(tail)))
    dz[ids[0]] -= 1e6 * q
    # The listed tokens' 1e6 (p - q) is past FP16's largest: an infinity of its sign.
    over = np.abs(dz) >= 65520
    assert (grad[0][over] == np.sign(dz[over]) * np.inf).all() and over.sum() == 3
    bad = np.abs(grad[0] - dz) > (HALF["f16"] + 8 * tol) * np.abs(dz) + 8 * tol * p * 1e6 + 2.0 ** -25
    assert not bad[~over].any()


def test_most_rows(gpu_lib):
    """WS_MAX_ROWS short rows of five kinds: each has the bits of the first of
    its kind and start, and the first rows are the oracle's."""
    import torch
    rows, V, few, k = lg.MAX_ROWS, 17, 5, 4
    rng = np.random.default_rng(2)
    z = _logits(rng, few, V)
    z[3, 4:] = -np.inf
    d = _dev()
    at = torch.arange(rows, device=d)
    kind = at % few
    mat = Matrix(np.zeros((0, V)), "bf16")
    mat.shape, mat.stride = (rows, V), V
    mat.view = torch.from_numpy(z).to(d).bfloat16()[kind].contiguous()
    head = Matrix(z[np.arange(40) % few], "bf16")
    ids, scores = make_teacher(rng, head.z[:few], k, ol.TAIL)
    targets, up = rng.integers(0, V, few), rng.normal(size=few)
    f = lambda *s: torch.zeros(s, dtype=torch.float32, device=d)  # noqa: E731
    teacher = teacher_entries(ids, scores)[kind].contiguous()
    tgt = torch.from_numpy(targets.astype(np.int32)).to(d)[kind].contiguous()
    g = _dev32(up)[kind].contiguous()
    lp, ent, st, loss, tail, dst = f(rows), f(rows), f(rows, 2), f(rows), f(rows), f(rows, 2)
    top = torch.zeros((rows, k, 2), dtype=torch.int32, device=d)
    grads = [torch.zeros((rows, V), dtype=torch.bfloat16, device=d) for _ in range(3)]
    r = mat.rows(1.1)
    for call in (lg.LogProbs(r, mat.view, targets=tgt, logprob=lp, entropy=ent, top_k=k, top=top,
                             stats=st),
                 lg.LogProbsGrad(r, mat.view, st, grads[0], targets=tgt, grad_logprob=g,
                                 entropy=ent, grad_entropy=g),
                 lg.Distill(r, mat.view, teacher, k, lg.DISTILL_TAIL, loss, stats=dst, tail=tail),
                 lg.DistillGrad(r, mat.view, teacher, k, lg.DISTILL_TAIL, dst, g, grads[1],
                                tail=tail),
                 lg.Distill(r, mat.view, teacher, k, lg.DISTILL_TAIL, loss, grad_loss=g,
                            grad_logits=grads[2])):
        call.run(torch.cuda.current_stream().cuda_stream)
    lead = at % 40                       # rows of 17 start alike every 8th
    for x in (lp, ent, st, top, loss, tail, dst, *grads):
        bits = x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)
        assert torch.equal(bits, bits[:40][lead])
    few_at = np.arange(40) % few
    check_logprobs(head, 1.1, targets[few_at], k=k, got={
        "logprob": lp[:40].cpu().numpy(), "entropy": ent[:40].cpu().numpy(),
        "stats": st[:40].cpu().numpy(), "top_id": top[:40, :, 1].cpu().numpy(),
        "top_score": top[:40].view(torch.float32)[:, :, 0].cpu().numpy()})
    a = run_logprobs_grad(head, 1.1, st[:40].cpu().numpy(), targets[few_at], up[few_at],
                          ent[:40].cpu().numpy(), up[few_at])
    b = run_distill(head, 1.1, ids[few_at], scores[few_at], ol.TAIL, up[few_at])
    c = run_distill(head, 1.1, ids[few_at], scores[few_at], ol.TAIL, up[few_at], separate=True)
    check_logprobs_grad(head, 1.1, targets[few_at], up[few_at], up[few_at])
    check_distill(head, 1.1, ids[few_at], scores[few_at], ol.TAIL, up[few_at])
    check_distill(head, 1.1, ids[few_at], scores[few_at], ol.TAIL, up[few_at], separate=True)
    for x, want in zip(grads, (a, c[1], b[1])):
        assert np.array_equal(x[:40].double().cpu().numpy(), want)


def test_longest_row(gpu_lib):
    """One row of WS_MAX_SCORES FP32 logits through every operator, against sums
    in 64 bits.  A thread adds 2^30 / 65,536 of them before it joins."""
    import torch
    V, k = 1 << 30, 8
    d = _dev()
    gen = torch.Generator(device=d)
    gen.manual_seed(9)
    z = torch.randn((1, V), device=d, generator=gen)
    hot = torch.tensor([3, V - 1, 1 << 29, V // 3, 77, V - 2, 12345678, V // 7], device=d)
    z[0, hot] += torch.arange(8, device=d) * 0.5 + 14.0
    step = 1 << 26
    m = float(z.max())
    total = u = 0.0
    for i in range(0, V, step):
        x = z[0, i:i + step].double() - m
        e = torch.exp(x)
        total += float(e.sum())
        u += float((e * x).sum())
        del x, e
    logsum = math.log(total)
    entropy = logsum - u / total
    order = hot[torch.argsort(z[0, hot], descending=True)]
    lp = {int(i): float(z[0, i]) - m - logsum for i in hot}
    f = lambda *s: torch.zeros(s, dtype=torch.float32, device=d)  # noqa: E731
    r = lg.make_rows(rows=1, vocab=V)
    got, ent, st, top = f(1), f(1), f(1, 2), torch.zeros((1, k, 2), dtype=torch.int32, device=d)
    target = torch.tensor([V - 1], dtype=torch.int32, device=d)
    lg.LogProbs(r, z, targets=target, logprob=got, entropy=ent, top_k=k, top=top, stats=st).run()
    torch.cuda.synchronize()
    tol = (V / 65536 + 100) * E + 8 * E * (1 + logsum)
    assert torch.equal(top[0, :, 1].long(), order) and float(st[0, 0]) == np.float32(m)
    assert abs(float(got) - lp[V - 1]) <= tol + 4 * E * abs(lp[V - 1])
    assert abs(float(st[0, 1]) - logsum) <= tol
    assert abs(float(ent) - entropy) <= 4 * tol * (1 + abs(logsum - entropy))
    scores = top.view(torch.float32)[0, :, 0].double().cpu().numpy()
    np.testing.assert_allclose(scores, [lp[int(i)] for i in order], atol=2 * tol + 100 * E)
    # Gradients, token by token: with upstreams of 1, p's relative error.
    rel = tol + 4 * E * (m + 8 + logsum) + 16 * E
    one = torch.ones(1, device=d)
    grad = torch.full((1, V), 7.0, device=d)
    lg.LogProbsGrad(r, z, st, grad, targets=target, grad_logprob=one).run()
    torch.cuda.synchronize()
    for i in range(0, V, step):
        want = -torch.exp(z[0, i:i + step].double() - m - logsum)
        if i <= V - 1 < i + step:
            want[V - 1 - i] += 1.0
        off = (grad[0, i:i + step].double() - want).abs() - rel * want.abs() - 8 * E * (want > 0)
        assert float(off.max()) <= 2.0 ** -126
        del want, off
    # The list holds part of the mass; the tail is the rest of the row.
    entries = top.clone()
    q = torch.arange(1, 9, device=d, dtype=torch.float64) / 48
    entries.view(torch.float32)[0, :, 0] = torch.log(q).float()
    q = torch.exp(entries.view(torch.float32)[0, :, 0].double())
    listed = sum(math.exp(v) for v in lp.values())
    tail, rest = math.log1p(-listed), 1.0 - float(q.sum())
    want = sum(float(w) * (math.log(w) - lp[int(i)]) for w, i in zip(q, order))
    want += rest * (math.log(rest) - tail)
    loss = f(1)
    lg.Distill(r, z, entries, k, lg.DISTILL_TAIL, loss, grad_loss=one, grad_logits=grad).run()
    torch.cuda.synchronize()
    assert abs(float(loss) - want) <= 4 * tol
    for i in range(0, V, step):
        p = torch.exp(z[0, i:i + step].double() - m - logsum)
        dz = p * (1.0 - rest / math.exp(tail))
        for w, j in zip(q, order):
            if i <= int(j) < i + step:
                dz[int(j) - i] = p[int(j) - i] - w
        off = (grad[0, i:i + step].double() - dz).abs() - 4 * rel * p - 8 * E * (p > 1e-4)
        assert float(off.max()) <= 2.0 ** -126
        del p, dz, off


def test_no_rows(gpu_lib):
    import torch
    z = torch.zeros((0, 50), device=_dev())
    r = lg.make_rows(rows=0, vocab=50)
    empty = torch.zeros((0,), device=_dev())
    lg.LogProbs(r, z, entropy=empty).run()
    lg.Distill(r, z, torch.zeros((0, 4, 2), dtype=torch.int32, device=_dev()), 4,
               lg.DISTILL_TAIL, empty).run()
    torch.cuda.synchronize()


def test_logprobs_offsets_past_32_bits(gpu_lib):
    """Rows whose elements start past 2^31 and bytes past 2^32."""
    import torch
    stride = 2 ** 30 + 24
    flat = torch.empty(2 * stride + 1000, dtype=torch.bfloat16, device=_dev())
    z = _logits(np.random.default_rng(6), 3, 1000)
    view = torch.as_strided(flat, (3, 1000), (stride, 1))
    view.copy_(torch.from_numpy(z).to(_dev()))
    mat = Matrix(np.zeros((0, 1000)), "bf16")
    mat.view, mat.stride, mat.shape = view, stride, (3, 1000)
    mat.z = view.double().cpu().numpy()
    check_logprobs(mat, 1.0, [1, 2, 3], k=6)


# ---------------------------------------------------------------------------
# Gradients of the log probabilities.


def _dev32(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(_dev())


def row_stats(mat, tau):
    """The statistics a forward call would leave, from the oracle."""
    out = np.array([ol.stats(z, _tau32(tau)) if not (np.isnan(z).any() or np.isposinf(z).any())
                    else (np.nan, np.nan) for z in mat.z])
    return out.reshape(-1, 2)


def grad_tol(z, tau, m, logsum, dtype, magnitude, p, V):
    """magnitude: sum of the absolute values of the terms multiplied by p;
    the terms themselves are part of `magnitude` where they stand alone."""
    t = np.where(np.isfinite(z), np.abs((z - m) / tau), 0.0)
    rel = 4 * E * (t + abs(logsum)) + 11 * E + _sum_tol(V)
    return (rel * p + 2.0 ** -126) * magnitude


def run_logprobs_grad(mat, tau, st, target=None, gl=None, ent=None, gh=None, ids=None, gk=None,
                      in_place=False, pad=0, shift=0):
    import torch
    rows, V = mat.shape
    d = _dev()
    kw = {}
    if target is not None:
        kw["targets"] = torch.from_numpy(np.asarray(target, dtype=np.int32)).to(d)
        kw["grad_logprob"] = _dev32(gl)
    if gh is not None:
        kw["entropy"] = _dev32(ent)
        kw["grad_entropy"] = _dev32(gh)
    if ids is not None:
        top = torch.full((rows, ids.shape[1], 2), 0x7fc00000, dtype=torch.int32, device=d)
        top[:, :, 1] = torch.from_numpy(np.asarray(ids, dtype=np.int32)).to(d)
        kw.update(top_k=ids.shape[1], top=top, grad_top=_dev32(gk))
    if in_place:
        out = mat
    else:
        out = Matrix(np.zeros((rows, V)), mat.dtype, pad, shift)
    call = lg.LogProbsGrad(mat.rows(tau), mat.view, _dev32(st), out.view,
                           grad_stride=out.stride, **kw)
    torch.cuda.synchronize()
    call.run()
    torch.cuda.synchronize()
    assert out.outside_untouched()
    return out.view.double().cpu().numpy()


def check_logprobs_grad(mat, tau, target=None, gl=None, gh=None, ids=None, gk=None, **kw):
    z = mat.z.copy()
    rows, V = z.shape
    st = row_stats(mat, tau)
    tau32 = _tau32(tau)
    ent = np.array([ol.entropy(ol.log_softmax(r, tau32)) for r in z])
    got = run_logprobs_grad(mat, tau, st, target, gl, ent, gh, ids, gk, **kw)
    f32 = lambda x: np.asarray(x, dtype=np.float32).astype(np.float64)  # noqa: E731
    for r in range(rows):
        t = int(target[r]) if target is not None else -1
        a = float(f32(gl)[r]) if target is not None else 0.0
        h = float(f32(gh)[r]) if gh is not None else 0.0
        i = ids[r] if ids is not None else ()
        g = f32(gk)[r] if ids is not None else ()
        want = ol.logprobs_grad(z[r], tau32, t, a, h, i, g)
        lp = ol.log_softmax(z[r], tau32)
        if np.isnan(want).any() or np.isneginf(lp).all():
            np.testing.assert_array_equal(got[r], want)
            continue
        p = np.exp(lp)
        bend = np.abs(np.where(p > 0, lp, 0.0)) + abs(ent[r])
        terms = abs(a) * (t >= 0) + sum(abs(x) for x in g) + abs(h) * (1 + bend)
        alone = np.zeros(V)
        if t >= 0:
            alone[t] += abs(a)
        for j, x in zip(i, g):
            if j >= 0:
                alone[j] += abs(x)
        tol = (grad_tol(z[r], tau32, st[r, 0], st[r, 1], mat.dtype, terms, p, V)
               + 4 * E * (alone + p * terms)) / tau32
        tol = tol + HALF[mat.dtype] * (np.abs(want) + tol) + SMALLEST[mat.dtype]
        assert_close(got[r], want, tol, f"gradient of row {r}")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V", [(1, 1), (3, 2), (4, 9), (3, 64), (2, 1000), (2, 4097),
                                    (1, 70001)])
def test_logprobs_grad_sizes(gpu_lib, dtype, rows, V):
    rng = np.random.default_rng(V)
    mat = Matrix(_logits(rng, rows, V), dtype)
    k = min(V, 32)
    ids = np.stack([rng.choice(V, k, replace=False) for _ in range(rows)])
    target = rng.integers(0, V, rows)
    ids[0, 0] = target[0]                            # the target among the alternatives
    check_logprobs_grad(mat, 1.0, target, rng.normal(size=rows))
    check_logprobs_grad(mat, 0.7, target, rng.normal(size=rows), rng.normal(size=rows), ids,
                        rng.normal(size=(rows, k)))
    check_logprobs_grad(mat, 2.0, gh=rng.normal(size=rows))
    check_logprobs_grad(mat, 1.0, ids=ids, gk=rng.normal(size=(rows, k)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift,gpad,gshift", [(0, 0, 5, 3), (3, 1, 3, 1), (3, 1, 0, 0),
                                                   (8, 8, 16, 8), (1, 0, 2, 1)])
def test_logprobs_grad_strides(gpu_lib, dtype, pad, shift, gpad, gshift):
    rng = np.random.default_rng(pad)
    mat = Matrix(_logits(rng, 5, 1003), dtype, pad, shift)
    check_logprobs_grad(mat, 1.0, rng.integers(0, 1003, 5), rng.normal(size=5),
                        rng.normal(size=5), pad=gpad, shift=gshift)
    check_logprobs_grad(mat, 1.0, rng.integers(0, 1003, 5), rng.normal(size=5), in_place=True)


def test_logprobs_grad_in_place_with_alternatives(gpu_lib):
    rng = np.random.default_rng(8)
    for V in (700, 40001):
        ids = np.stack([rng.choice(V, 8, replace=False) for _ in range(4)])
        mat = Matrix(_logits(rng, 4, V), "bf16", 1, 1)
        check_logprobs_grad(mat, 1.0, ids[:, 0], rng.normal(size=4), rng.normal(size=4), ids,
                            rng.normal(size=(4, 8)), in_place=True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [6, 300, 9001])
def test_logprobs_grad_special_rows(gpu_lib, dtype, V):
    z = special_rows(V, dtype)
    rng = np.random.default_rng(V)
    rows = len(z)
    target = rng.integers(0, V, rows)
    ids = np.stack([rng.choice(V, 4, replace=False) for _ in range(rows)])
    check_logprobs_grad(Matrix(z, dtype), 1.0, target, rng.normal(size=rows),
                        rng.normal(size=rows), ids, rng.normal(size=(rows, 4)))


def test_logprobs_grad_indices_outside_and_absent(gpu_lib):
    rng = np.random.default_rng(2)
    mat = Matrix(_logits(rng, 6, 400), "f32")
    ids = np.array([[1, 1, 1], [-1, 5, -1], [400, 1, 2], [3, -2, 4], [7, 8, 9], [-1, -1, -1]])
    check_logprobs_grad(mat, 1.0, [1, -1, 0, 1, 400, -1], rng.normal(size=6), None, ids,
                        rng.normal(size=(6, 3)))


def test_index_outside_a_row_without_a_distribution(gpu_lib):
    """An index outside the row makes the whole gradient NaN, in a row of -inf
    only as in any other."""
    z = np.full((3, 40), -np.inf)
    z[2] = 1.0
    check_logprobs_grad(Matrix(z, "f32"), 1.0, [40, 3, 41], np.ones(3))
    ids = np.array([[1, 40], [1, 2], [-3, 2]])
    scores = np.log(np.full((3, 2), 0.25))
    for mode in (ol.RENORM, ol.TAIL):
        mat = Matrix(z, "f32")
        check_distill(mat, 1.0, ids, scores, mode, np.ones(3))
        _, grad, _, _ = run_distill(mat, 1.0, ids, scores, mode, np.ones(3))
        _, apart, _, _ = run_distill(mat, 1.0, ids, scores, mode, np.ones(3), separate=True)
        for got in (grad, apart):
            assert np.isnan(got[0]).all() and (got[1] == 0).all() and np.isnan(got[2]).all()


def test_logprobs_gradient_against_differences(gpu_lib):
    """The gradient against differences of the forward operator itself: FP32
    outputs carry about 1e-6, so a step of 1e-2 leaves 1e-4 of noise and the
    quotient's own h^2 f''' / 6 < 1e-4 of truncation."""
    rng = np.random.default_rng(12)
    V, h = 24, 1e-2
    base = rng.normal(size=V)
    z = np.concatenate([np.stack([base + h * (np.arange(V) == j), base - h * (np.arange(V) == j)])
                        for j in range(V)])
    got = run_logprobs(Matrix(z, "f32"), 1.0, np.full(2 * V, 5))
    f = 0.8 * got["logprob"].astype(np.float64) - 0.3 * got["entropy"]
    want = (f[0::2] - f[1::2]) / (2 * h)
    mat = Matrix(base[None], "f32")
    fwd = run_logprobs(mat, 1.0, [5])
    grad = run_logprobs_grad(mat, 1.0, fwd["stats"], [5], [0.8], fwd["entropy"], [-0.3])
    np.testing.assert_allclose(grad[0], want, atol=2e-4)


# ---------------------------------------------------------------------------
# Distillation.


def teacher_entries(ids, scores):
    import torch
    top = torch.empty(ids.shape + (2,), dtype=torch.int32, device=_dev())
    top[:, :, 0] = _dev32(scores).view(torch.int32)
    top[:, :, 1] = torch.from_numpy(np.asarray(ids, dtype=np.int32)).to(_dev())
    return top


def make_teacher(rng, z, k, mode):
    """k entries a row from a noisy copy of the logits: log probabilities."""
    ids, scores = [], []
    for row in z:
        y = np.where(np.isfinite(row), row, -30.0) + rng.normal(size=len(row))
        y = np.clip(y, -100.0, 100.0)
        i = ol.best(y, k)
        lp = ol.log_softmax(y, 1.0)
        ids.append(i)
        scores.append(lp[i] + (0.0 if mode == ol.TAIL else 3.0))
    return np.array(ids), np.array(scores, dtype=np.float32)


def run_distill(mat, tau, ids, scores, mode, g=None, in_place=False, pad=0, shift=0,
                separate=False):
    import torch
    rows, V = mat.shape
    d = _dev()
    loss = torch.full((rows,), -5.0, dtype=torch.float32, device=d)
    stats = torch.zeros((rows, 2), dtype=torch.float32, device=d)
    tail = torch.zeros((rows,), dtype=torch.float32, device=d) if mode == ol.TAIL else None
    top = teacher_entries(ids, scores)
    k = ids.shape[1]
    gl = _dev32(g) if g is not None else None
    out = None
    if g is not None:
        out = mat if in_place else Matrix(np.zeros((rows, V)), mat.dtype, pad, shift)
    r = mat.rows(tau)
    if separate or g is None:
        calls = [lg.Distill(r, mat.view, top, k, mode, loss, stats=stats, tail=tail)]
        if separate:
            calls.append(lg.DistillGrad(r, mat.view, top, k, mode, stats, gl, out.view, tail=tail,
                                        grad_stride=out.stride))
    else:
        calls = [lg.Distill(r, mat.view, top, k, mode, loss, grad_loss=gl, grad_logits=out.view,
                            grad_stride=out.stride)]
    torch.cuda.synchronize()
    for c in calls:
        c.run()
    torch.cuda.synchronize()
    if out is not None:
        assert out.outside_untouched()
    grad = out.view.double().cpu().numpy() if out is not None else None
    return loss.cpu().numpy(), grad, stats.cpu().numpy(), tail


def check_distill(mat, tau, ids, scores, mode, g=None, **kw):
    z = mat.z.copy()
    rows, V = z.shape
    loss, grad, st, tail_got = run_distill(mat, tau, ids, scores, mode, g, **kw)
    tau32 = _tau32(tau)
    scores = np.asarray(scores, dtype=np.float32).astype(np.float64)
    g64 = np.asarray(g, dtype=np.float32).astype(np.float64) if g is not None else np.ones(rows)
    for r in range(rows):
        want, dz, tail = ol.distill(z[r], tau32, scores[r], ids[r], mode, g64[r])
        lp = ol.log_softmax(z[r], tau32)
        m, logsum = ol.stats(z[r], tau32)
        if np.isnan(want):
            assert np.isnan(loss[r])
        else:
            q, logq, rest = ol.teacher_weights(scores[r], ids[r], V, mode)
            zk = z[r][np.where(ids[r] < 0, 0, ids[r])]
            zk = np.where(np.isfinite(zk), zk, m if np.isfinite(m) else 0.0)
            ls = logsum if np.isfinite(logsum) else 0.0
            d = np.abs((zk - (m if np.isfinite(m) else 0.0)) / tau32)
            # One inverse temperature rounded to FP32, one log sum for all.
            tol = (q * (2 * E * d)).sum() + (q.sum() + 2 * rest) * (_sum_tol(V) + 8 * E * (1 + abs(ls)))
            if rest > 0 and np.isfinite(tail):
                tol += 8 * E * rest * abs(tail)
            tol += 2 * E * abs(want if np.isfinite(want) else 0.0) + 1e-37
            assert_close(loss[r], want, tol, f"loss of row {r}")
        if g is None:
            continue
        if np.isnan(dz).any() or np.isneginf(lp).all():
            np.testing.assert_array_equal(grad[r], dz)
            continue
        p = np.exp(lp)
        q, logq, rest = ol.teacher_weights(scores[r], ids[r], V, mode)
        alone = np.zeros(V)
        np.add.at(alone, ids[r][ids[r] >= 0], q[ids[r] >= 0])
        mass = q.sum() + rest
        weight = p * mass
        tail_err = 0.0
        if mode == ol.TAIL and rest > 0 and np.isfinite(tail):
            # Unlisted tokens: p_j / p_t (M p_t - q_t), both sums in the quotient.
            listed = np.isin(np.arange(V), ids[r])
            with np.errstate(over="ignore"):
                share = np.exp(np.where(listed, -np.inf, lp - tail))
            weight = np.where(listed, weight, share * (mass * np.exp(tail) + rest))
            tail_err = 2 * _sum_tol(V) + 8 * E * (1 + abs(tail))
        tol = grad_tol(z[r], tau32, m, logsum, mat.dtype, weight, 1.0, V)
        tol = tol + weight * tail_err + 4 * E * (alone + weight) + 2.0 ** -126 * mass
        tol = tol * abs(g64[r]) / tau32
        tol = tol + HALF[mat.dtype] * (np.abs(dz) + tol) + SMALLEST[mat.dtype]
        assert_close(grad[r], dz, tol, f"gradient of row {r}")


@pytest.mark.parametrize("mode", [ol.RENORM, ol.TAIL])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V,k", [(1, 1, 1), (3, 2, 1), (2, 9, 9), (4, 65, 3), (3, 1000, 5),
                                      (2, 4097, 128), (2, 21843, 64), (1, 70001, 33)])
def test_distill_sizes(gpu_lib, mode, dtype, rows, V, k):
    rng = np.random.default_rng(V + k)
    z = _logits(rng, rows, V)
    mat = Matrix(z, dtype)
    ids, scores = make_teacher(rng, mat.z, k, mode)
    g = rng.random(rows) * 64
    check_distill(mat, 1.0, ids, scores, mode)
    check_distill(mat, 1.4, ids, scores, mode, g)
    check_distill(mat, 1.4, ids, scores, mode, g, separate=True)
    check_distill(mat, 1.0, ids, scores, mode, g, in_place=True)


@pytest.mark.parametrize("mode", [ol.RENORM, ol.TAIL])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,shift,gpad,gshift", [(0, 0, 5, 3), (3, 1, 3, 1), (3, 1, 0, 0),
                                                   (8, 8, 16, 8)])
def test_distill_strides(gpu_lib, mode, dtype, pad, shift, gpad, gshift):
    rng = np.random.default_rng(pad + 10)
    V = 1503
    mat = Matrix(_logits(rng, 5, V), dtype, pad, shift, marker=1e4)
    ids, scores = make_teacher(rng, mat.z, 17, mode)
    ids[0, 0] = V - 1
    ids[1, 3] = 0
    check_distill(mat, 1.0, ids, scores, mode, rng.random(5) * 9, pad=gpad, shift=gshift)
    check_distill(mat, 1.0, ids, scores, mode, rng.random(5) * 9, separate=True, in_place=True)


@pytest.mark.parametrize("mode", [ol.RENORM, ol.TAIL])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [6, 300, 9001])
def test_distill_special_rows(gpu_lib, mode, dtype, V):
    z = special_rows(V, dtype)
    rng = np.random.default_rng(V)
    ids, scores = make_teacher(rng, z, 4, mode)
    mat = Matrix(z, dtype)
    check_distill(mat, 1.0, ids, scores, mode, rng.random(len(z)))
    check_distill(Matrix(z, dtype), 1.0, ids, scores, mode, rng.random(len(z)), separate=True)


@pytest.mark.parametrize("mode", [ol.RENORM, ol.TAIL])
@pytest.mark.parametrize("dtype,V", [("f32", 900), ("f32", 20003), ("f32", 50001), ("f16", 5),
                                     ("bf16", 9001), ("bf16", 40001), ("bf16", 70001),
                                     ("bf16", 131072), ("bf16", 131073)])
def test_distill_many_rows(gpu_lib, mode, dtype, V):
    """Enough rows for a workgroup to hold a whole row, of each size of
    workgroup, up to and past what it holds."""
    import torch
    rng = np.random.default_rng(V)
    rows, few = 130, 5
    z = np.broadcast_to(_logits(rng, few, V)[np.arange(rows) % few], (rows, V))
    mat = Matrix(z, dtype, 1 if V == 9001 else 0, 3 if V == 9001 else 0)
    k = min(V, 40)
    ids, scores = make_teacher(rng, mat.z[:few], k, mode)
    ids, scores = ids[np.arange(rows) % few].copy(), scores[np.arange(rows) % few]
    ids[3, 0] = -1
    ids[4, 0] = V - 1
    ids[4, 1:] = np.where(ids[4, 1:] == V - 1, -1, ids[4, 1:])
    g = np.arange(rows) + 1.0
    loss, grad, _, _ = run_distill(mat, 1.2, ids, scores, mode, g)
    # The first rows against the oracle, the others against the same row among them.
    small = Matrix(z[:few], dtype)
    check_distill(small, 1.2, ids[:few], scores[:few], mode, g[:few])
    check_distill(mat, 1.2, ids, scores, mode, g, in_place=True) if V < 10000 else None
    sub, subgrad, _, _ = run_distill(small, 1.2, ids[:few], scores[:few], mode, g[:few])
    half = HALF[dtype]
    np.testing.assert_allclose(loss[:few], sub, rtol=2 * _sum_tol(V), atol=2 * _sum_tol(V) * 20)
    for r in range(few):
        peak = np.abs(subgrad[r]).max()
        # Two sums of one row in different orders, then two roundings.
        np.testing.assert_allclose(grad[r], subgrad[r], rtol=2.1 * half + 4 * _sum_tol(V),
                                   atol=8 * _sum_tol(V) * peak + 2 * SMALLEST[dtype])
    for r in (few + 1, rows - 1):
        np.testing.assert_allclose(loss[r], loss[r % few] if r % few not in (3, 4) else loss[r],
                                   rtol=1e-6)


@pytest.mark.parametrize("mode", [ol.RENORM, ol.TAIL])
@pytest.mark.parametrize("dtype,V", [("f32", 300), ("f16", 2500), ("bf16", 9001), ("bf16", 40000)])
def test_distill_many_special_rows(gpu_lib, mode, dtype, V):
    """The special rows among enough others for a workgroup to hold a row."""
    rng = np.random.default_rng(V + 1)
    special = special_rows(V, dtype)
    z = np.concatenate([special] + [_logits(rng, 130 - len(special), V)])
    ids, scores = make_teacher(rng, z[:20], 4, mode)
    ids, scores = np.tile(ids, (7, 1))[:130], np.tile(scores, (7, 1))[:130]
    mat = Matrix(z, dtype)
    check_distill(mat, 1.0, ids, scores, mode, rng.random(130))


@pytest.mark.parametrize("mode", [ol.RENORM, ol.TAIL])
@pytest.mark.parametrize("dtype,rows,V,pad,shift", [
    ("f32", 6, 15001, 0, 0), ("f32", 6, 30001, 3, 2), ("f32", 6, 65536, 0, 0),
    ("f32", 5, 65530, 3, 1), ("f16", 6, 30001, 1, 1), ("f16", 6, 60001, 0, 0),
    ("f16", 80, 131072, 0, 0), ("bf16", 6, 30001, 0, 0), ("bf16", 6, 60001, 5, 3),
    ("bf16", 81, 131064, 1, 0)])
def test_distill_held_rows_against_the_oracle(gpu_lib, mode, dtype, rows, V, pad, shift):
    """Loss and gradient of every row and token of the kernel that holds a row,
    with four, eight and sixteen waves and rows that fill them."""
    rng = np.random.default_rng(V + mode)
    few = min(rows, 6)
    z = _logits(rng, few, V)
    z[2, rng.random(V) < 0.9] = -np.inf
    at = np.arange(rows) % few
    mat = Matrix(z[at], dtype, pad, shift)
    ids, scores = make_teacher(rng, mat.z[:few], 50, mode)
    ids[1, 4:9] = -1
    ids[3, 1] = V - 1 if V - 1 not in ids[3] else ids[3, 1]
    check_distill(mat, 1.3, ids[at], scores[at], mode, (rng.random(rows) + 0.5) * 1e3,
                  pad=pad, shift=shift)


@pytest.mark.parametrize("mode", [ol.RENORM, ol.TAIL])
@pytest.mark.parametrize("dtype,V", [("f32", 900), ("f32", 20004), ("f32", 50004), ("f16", 40000),
                                     ("f16", 100008), ("bf16", 9008), ("bf16", 131072)])
def test_distill_rows_that_repeat_have_the_same_bits(gpu_lib, mode, dtype, V):
    """130 rows of five kinds at starts that lie alike: loss and gradient of
    every row are those of its kind's first, bit for bit, in place as well."""
    rng = np.random.default_rng(V)
    rows, few = 130, 5
    at = np.arange(rows) % few
    mat = Matrix(_logits(rng, few, V)[at], dtype)
    ids, scores = make_teacher(rng, mat.z[:few], 40, mode)
    ids[3, 0] = -1
    g = (np.arange(few) + 1.0)[at]
    loss, grad, _, _ = run_distill(mat, 1.2, ids[at], scores[at], mode, g)
    small = Matrix(mat.z[:few], dtype)
    check_distill(small, 1.2, ids, scores, mode, g[:few])
    here, dhere, _, _ = run_distill(mat, 1.2, ids[at], scores[at], mode, g, in_place=True)
    for l, d in ((loss, grad), (here, dhere)):
        assert (l == loss[at]).all()
        for r in range(rows):
            assert np.array_equal(d[r], grad[r % few])


@pytest.mark.parametrize("mode", [ol.RENORM, ol.TAIL])
@pytest.mark.parametrize("dtype,rows,V", [("f32", 6, 5000), ("bf16", 80, 70001), ("f16", 4, 90001)])
def test_distill_one_call_against_two(gpu_lib, mode, dtype, rows, V):
    """Loss and gradient of one call against those of ws_distill and then
    ws_distill_grad: each is within its tolerance of the formula, so the two are
    within twice that of each other; statistics in FP32 between the two calls
    are half a step of each more."""
    rng = np.random.default_rng(15 + V)
    few = min(rows, 6)
    at = np.arange(rows) % few
    mat = Matrix(_logits(rng, few, V)[at], dtype)
    ids, scores = make_teacher(rng, mat.z[:few], 40, mode)
    g = rng.random(rows)
    one, done, _, _ = run_distill(mat, 1.0, ids[at], scores[at], mode, g)
    two, dtwo, st, _ = run_distill(mat, 1.0, ids[at], scores[at], mode, g, separate=True)
    listed = np.zeros(V, dtype=bool)
    for r in range(rows):
        z, i = mat.z[r], ids[r % few]
        want, dz, tail = ol.distill(z, 1.0, scores[r % few].astype(np.float64), i, mode)
        q, _, rest = ol.teacher_weights(scores[r % few].astype(np.float64), i, V, mode)
        m, logsum = ol.stats(z, 1.0)
        step = _sum_tol(V) + 8 * E * (1 + logsum)
        tol = (q * 2 * E * (m - z[i])).sum() + (q.sum() + 2 * rest) * step + 2 * E * abs(want)
        tol += 8 * E * rest * abs(tail) if mode == ol.TAIL else 0.0
        assert abs(float(one[r]) - float(two[r])) <= 2 * tol
        lp = z - m - logsum
        listed[:] = False
        listed[i] = True
        weight = np.exp(lp) * (q.sum() + rest)
        if mode == ol.TAIL:
            share = np.exp(np.where(listed, -np.inf, lp - tail))
            weight = np.where(listed, weight, share * (np.exp(tail) + rest))
            step += 2 * _sum_tol(V) + 8 * E * (1 + abs(tail))
        alone = np.zeros(V)
        alone[i] = q
        tol = (4 * E * (m - z + logsum) + 11 * E + step) * weight + 4 * E * (alone + weight)
        tol = (tol + 2.0 ** -126) * g[r]
        tol = tol + HALF[dtype] * (np.abs(dz) * g[r] + tol) + SMALLEST[dtype]
        off = np.abs(done[r] - dtwo[r]) - 2 * tol
        assert (off <= 0).all(), f"row {r}, token {off.argmax()}: {off.max()} past the tolerance"


@pytest.mark.parametrize("mode", [ol.RENORM, ol.TAIL])
def test_distill_entries(gpu_lib, mode):
    """Absent entries, none at all, the same token twice, scores of -inf,
    indices outside the row, every token listed, a teacher certain of one."""
    rng = np.random.default_rng(21)
    V = 8
    inf = np.inf
    ids = np.array([[0, -1, 3, -1], [-1, -1, -1, -1], [2, 2, 5, 2], [1, 4, 6, 7], [8, 1, 2, 3],
                    [-7, 1, 2, 3], [5, -1, -1, -1], [3, 3, 3, 3], [0, 1, 2, 3]])
    scores = np.log(np.array([[.5, .9, .2, .9], [.1, .1, .1, .1], [.2, .3, .1, .05],
                              [.4, .1, .1, .1], [.1, .1, .1, .1], [.1, .1, .1, .1],
                              [1.0, 1, 1, 1], [.25, .25, .25, .25], [.5, .3, .1, .1]]))
    scores[3, 2] = -inf
    z = rng.normal(size=(9, V))
    for dtype in ("f32", "bf16"):
        mat = Matrix(z, dtype)
        check_distill(mat, 1.0, ids, scores, mode, np.ones(9))
        check_distill(mat, 1.0, ids, scores, mode, np.ones(9), separate=True)
    every = np.tile(np.arange(V), (2, 1))
    lp = np.stack([ol.log_softmax(rng.normal(size=V), 1.0) for _ in range(2)])
    check_distill(Matrix(z[:2], "f32"), 1.0, every, lp, mode, np.ones(2))
    none = np.full((2, 3), -inf)
    check_distill(Matrix(z[:2], "f32"), 1.0, every[:, :3], none, mode, np.ones(2))


def test_distill_tail_far_below_the_listed_tokens(gpu_lib):
    """A student certain of the listed tokens: the tail's probability is far
    below what a difference of FP32 sums could hold."""
    V = 3000
    z = np.random.default_rng(1).normal(size=(3, V))
    z[:, 7] += np.array([30.0, 80.0, 300.0])
    ids = np.tile(np.array([[7, 100]]), (3, 1))
    scores = np.tile(np.log(np.array([[0.9, 0.05]])), (3, 1))
    check_distill(Matrix(z, "f32"), 1.0, ids, scores, ol.TAIL, np.ones(3))
    check_distill(Matrix(z, "f32"), 1.0, ids, scores, ol.TAIL, np.ones(3), separate=True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,V", [(40, 1000), (70, 40001), (30, 70001)])
def test_distill_rows_masked_to_fewer_tokens_than_are_listed(gpu_lib, dtype, rows, V):
    """As a grammar leaves them: 12 allowed tokens, teacher entries from
    ws_logprobs with K = 20, so the list holds all of the mass and 1 - sum q is
    rounding.  The loss is the divergence over the allowed tokens and the
    gradient of every other token 0, whichever value masks them."""
    rng = np.random.default_rng(V)
    low = {"f32": -3.4028234663852886e38, "f16": -65504.0, "bf16": -3.3895313892515355e38}[dtype]
    for mask in (-np.inf, low):
        zt, zs = np.full((rows, V), mask), np.full((rows, V), mask)
        allowed = np.stack([rng.choice(V, 12, replace=False) for _ in range(rows)])
        np.put_along_axis(zt, allowed, rng.normal(size=(rows, 12)) * 3, 1)
        np.put_along_axis(zs, allowed, rng.normal(size=(rows, 12)) * 3, 1)
        top = run_logprobs(Matrix(zt, dtype), 1.0, None, k=20)
        ids, scores = top["top_id"], top["top_score"]
        student = Matrix(zs, dtype)
        g = np.ones(rows)
        for separate in (False, True):
            loss, grad, st, _ = run_distill(student, 1.0, ids, scores, ol.TAIL, g,
                                            separate=separate)
            assert np.isfinite(loss).all()
            for r in range(rows):
                at = ids[r][:12]
                assert set(at) == set(allowed[r])
                q = np.exp(scores[r][:12].astype(np.float64))
                z = student.z[r][at]
                lp = ol.log_softmax(z, 1.0)
                m, logsum = ol.stats(z, 1.0)
                want = (q * (np.log(q) - lp)).sum()
                tol = (q * (2 * E * (m - z))).sum() + q.sum() * (_sum_tol(V) + 8 * E * (1 + logsum))
                assert abs(loss[r] - want) <= tol + 2 * E * abs(want)
                p, mass = np.exp(lp), q.sum()
                dz = mass * p - q
                tol = (grad_tol(z, 1.0, m, logsum, dtype, mass, p, V) + 4 * E * (q + mass * p))
                tol = tol + HALF[dtype] * (np.abs(dz) + tol) + SMALLEST[dtype]
                assert_close(grad[r][at], dz, tol, f"gradient of row {r}")
                assert not np.delete(grad[r], at).any()


@pytest.mark.parametrize("mode", [ol.RENORM, ol.TAIL])
@pytest.mark.parametrize("dtype,V,repeat", [("f32", 300, 1), ("f16", 2500, 9), ("bf16", 70001, 1),
                                            ("bf16", 70001, 6), ("f32", 9, 1)])
def test_distill_special_rows_without_entries(gpu_lib, mode, dtype, V, repeat):
    """A row that holds a NaN or +inf has a NaN loss and gradient whatever is
    listed: nothing, or tokens of probability 0 only; in a held row, a whole
    one and one in parts."""
    z = np.tile(special_rows(V, dtype), (repeat, 1))
    rows = len(z)
    held_bad = np.isnan(z).any(1) | np.isposinf(z).any(1)
    assert held_bad.sum() == 3 * repeat
    absent = np.full((rows, 9), -1)
    zero = np.tile(np.arange(9), (rows, 1))
    for ids, scores in ((absent, np.zeros((rows, 9))), (zero, np.full((rows, 9), -np.inf))):
        for kw in ({}, {"separate": True}):
            mat = Matrix(z, dtype)
            loss, grad, _, _ = run_distill(mat, 1.0, ids, scores, mode, np.ones(rows), **kw)
            assert (np.isnan(loss) == held_bad).all()
            assert (np.isnan(grad).any(1) == held_bad).all()
            assert np.isnan(grad[held_bad]).all()
            if mode == ol.RENORM:
                assert (loss[~held_bad] == 0).all() and (grad[~held_bad] == 0).all()
        check_distill(Matrix(z[:16], dtype), 1.0, ids[:16], scores[:16], mode, np.ones(16))


def test_distill_teacher_nearly_certain_of_one_token(gpu_lib):
    """A q_t far below FP32's half step at 1, against a p_t of its size or
    below: what 1 - sum q keeps in FP64 shows in the gradient."""
    V = 40
    z = np.zeros((3, V))
    z[:, 4] = [24.0, 30.0, 27.0]
    ids = np.full((3, 1), 4)
    scores = np.array([[-1e-9], [-1e-10], [-1e-10]])
    for kw in ({}, {"separate": True}):
        check_distill(Matrix(z, "f32"), 1.0, ids, scores, ol.TAIL, np.ones(3), **kw)


def test_distill_gradient_against_differences(gpu_lib):
    """As for the log probabilities: noise 1e-4, truncation below 1e-4."""
    rng = np.random.default_rng(14)
    V, h = 24, 1e-2
    base = rng.normal(size=V)
    ids, scores = make_teacher(rng, base[None], 6, ol.TAIL)
    z = np.concatenate([np.stack([base + h * (np.arange(V) == j), base - h * (np.arange(V) == j)])
                        for j in range(V)])
    for mode in (ol.RENORM, ol.TAIL):
        loss, _, _, _ = run_distill(Matrix(z, "f32"), 1.0, np.tile(ids, (2 * V, 1)),
                                    np.tile(scores, (2 * V, 1)), mode)
        want = (loss[0::2].astype(np.float64) - loss[1::2]) / (2 * h)
        _, grad, _, _ = run_distill(Matrix(base[None], "f32"), 1.0, ids, scores, mode, np.ones(1))
        np.testing.assert_allclose(grad[0], want, atol=2e-4)


def test_distill_in_one_call_and_in_two_agree(gpu_lib):
    """One call and loss-then-gradient give the gradient of the same row to
    within the two calls' rounded statistics."""
    rng = np.random.default_rng(15)
    mat = Matrix(_logits(rng, 6, 5000), "f32")
    ids, scores = make_teacher(rng, mat.z, 40, ol.TAIL)
    g = rng.random(6)
    check_distill(mat, 1.0, ids, scores, ol.TAIL, g)
    check_distill(mat, 1.0, ids, scores, ol.TAIL, g, separate=True)


# ---------------------------------------------------------------------------
# The operators together, and how they are called.


def test_teacher_to_student_run(gpu_lib):
    """As used: the teacher's alternatives from ws_logprobs are, in place, the
    entries ws_distill takes; the student's loss and gradient follow, then the
    student's own log probabilities and their gradient."""
    import torch
    rng = np.random.default_rng(16)
    rows, V, k, tau = 12, 4001, 24, 1.5
    teacher = Matrix(_logits(rng, rows, V), "bf16")
    student = Matrix(teacher.z + rng.normal(size=(rows, V)), "bf16")
    got = check_logprobs(teacher, tau, None, k=k)
    top = got["device"]["top"]
    loss = torch.empty(rows, device=_dev())
    grad = torch.empty(rows, V, dtype=torch.bfloat16, device=_dev())
    g = np.full(rows, 1.0 / rows)
    call = lg.Distill(student.rows(tau), student.view, top, k, lg.DISTILL_TAIL, loss,
                      grad_loss=_dev32(g), grad_logits=grad)
    call.run(torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    ids, scores = got["top_id"], got["top_score"]
    want, wgrad, _, _ = run_distill(student, tau, ids, scores, ol.TAIL, g)
    np.testing.assert_array_equal(loss.cpu().numpy(), want)
    np.testing.assert_array_equal(grad.double().cpu().numpy(), wgrad)
    check_distill(student, tau, ids, scores, ol.TAIL, g)
    fwd = check_logprobs(student, tau, ids[:, 0], k=4)
    check_logprobs_grad(student, tau, ids[:, 0], g, 0.01 * g, fwd["top_id"], np.zeros((rows, 4)))


def test_student_trains_towards_the_teacher(gpu_lib):
    """An update along the gradient is the gradient's own first-order change
    of the loss (not how far it falls: the slope)."""
    rng = np.random.default_rng(18)
    z = _logits(rng, 4, 300)
    ids, scores = make_teacher(rng, z, 10, ol.TAIL)
    loss, grad, _, _ = run_distill(Matrix(z, "f32"), 1.0, ids, scores, ol.TAIL, np.ones(4))
    h = 1e-2 / np.abs(grad).max()
    up = run_distill(Matrix(z + h * grad, "f32"), 1.0, ids, scores, ol.TAIL)[0]
    down = run_distill(Matrix(z - h * grad, "f32"), 1.0, ids, scores, ol.TAIL)[0]
    slope = (up.astype(np.float64) - down) / (2 * h)
    np.testing.assert_allclose(slope, (grad ** 2).sum(1), rtol=2e-3, atol=2e-3)


def _all_calls(seed, rows, V, dtype):
    """Every operator bound on its own buffers, with what they write."""
    import torch
    rng = np.random.default_rng(seed)
    mat = Matrix(_logits(rng, rows, V), dtype)
    d = _dev()
    k = min(V, 16)
    ids, scores = make_teacher(rng, mat.z, k, ol.TAIL)
    top = torch.zeros((rows, k, 2), dtype=torch.int32, device=d)
    f = lambda *s: torch.zeros(s, dtype=torch.float32, device=d)  # noqa: E731
    targets = torch.from_numpy(rng.integers(0, V, rows).astype(np.int32)).to(d)
    lp, ent, st, loss, dst, tail = f(rows), f(rows), f(rows, 2), f(rows), f(rows, 2), f(rows)
    loss2 = f(rows)
    g1, g2, g3 = (torch.zeros((rows, V), dtype=_torch_type(dtype), device=d) for _ in range(3))
    teacher = teacher_entries(ids, scores)
    up = _dev32(rng.normal(size=rows))
    r = mat.rows(1.1)
    calls = [lg.LogProbs(r, mat.view, targets=targets, logprob=lp, entropy=ent, top_k=k, top=top,
                         stats=st),
             lg.LogProbsGrad(r, mat.view, st, g1, targets=targets, grad_logprob=up, entropy=ent,
                             grad_entropy=up, top_k=k, top=top, grad_top=_dev32(
                                 rng.normal(size=(rows, k)))),
             lg.Distill(r, mat.view, teacher, k, lg.DISTILL_TAIL, loss, stats=dst, tail=tail),
             lg.DistillGrad(r, mat.view, teacher, k, lg.DISTILL_TAIL, dst, up, g2, tail=tail),
             lg.Distill(r, mat.view, teacher, k, lg.DISTILL_TAIL, loss2, grad_loss=up,
                        grad_logits=g3)]
    return mat, calls, [lp, ent, st, top, loss, dst, tail, loss2, g1, g2, g3]


def _bits(tensors):
    import torch
    return [t.contiguous().view(torch.uint8).cpu().numpy().copy() for t in tensors]


@pytest.mark.parametrize("rows,V", [(3, 700), (2, 40001), (40, 9000)])
def test_captured_and_replayed(gpu_lib, rows, V):
    """The whole run in one graph, replayed on changed logits with eager work
    and synchronisation in between: each replay's bits are the eager ones."""
    import torch
    mat, calls, outs = _all_calls(31, rows, V, "bf16")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for c in calls:
            c.run(torch.cuda.current_stream().cuda_stream)
    rng = np.random.default_rng(5)
    for _ in range(4):
        mat.view.copy_(torch.from_numpy(_logits(rng, rows, V)).to(_dev()))
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = _bits(outs)
        for o in outs:
            o.zero_()
        for c in calls:
            c.run(torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        for a, b in zip(replayed, _bits(outs)):
            np.testing.assert_array_equal(a, b)


def test_two_streams_at_once(gpu_lib):
    """Two sets of bound calls (a workspace each) in flight on two streams
    give what each gives alone."""
    import torch
    sets = [_all_calls(41, 2, 60001, "bf16"), _all_calls(42, 3, 30011, "f32")]
    alone = []
    for _, calls, outs in sets:
        for c in calls:
            c.run()
        torch.cuda.synchronize()
        alone.append(_bits(outs))
        for o in outs:
            o.zero_()
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(5):
        for (_, calls, _), s in zip(sets, streams):
            for c in calls:
                c.run(s.cuda_stream)
    torch.cuda.synchronize()
    for (_, _, outs), want in zip(sets, alone):
        for a, b in zip(_bits(outs), want):
            np.testing.assert_array_equal(a, b)


def test_two_captured_graphs_with_a_workspace_each(gpu_lib):
    import torch
    sets = [_all_calls(51, 2, 50021, "f16"), _all_calls(52, 1, 65536, "bf16")]
    graphs, alone = [], []
    for _, calls, outs in sets:
        for c in calls:
            c.run()
        torch.cuda.synchronize()
        alone.append(_bits(outs))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for c in calls:
                c.run(torch.cuda.current_stream().cuda_stream)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in sets]
    for _, _, outs in sets:
        for o in outs:
            o.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, _, outs), want in zip(sets, alone):
        for a, b in zip(_bits(outs), want):
            np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("dtype,rows,V,gap", [("f32", 5, 1003, 3), ("bf16", 5, 1003, 0),
                                              ("f16", 90, 2000, 5), ("bf16", 3, 70001, 1)])
def test_gradient_rows_between_the_logits_rows(gpu_lib, dtype, rows, V, gap):
    """One buffer that holds a row of logits and a row of gradients in turn:
    the bits of a gradient apart from them, and the logits left as they were."""
    import torch
    rng = np.random.default_rng(V + gap)
    z = _logits(rng, rows, V)
    pad = V + 2 * gap
    apart, both = Matrix(z, dtype, pad), Matrix(z, dtype, pad)
    start = V + gap
    grad = torch.as_strided(both.flat, (rows, V), (both.stride, 1), start)
    ids, scores = make_teacher(rng, apart.z, 9, ol.TAIL)
    top = teacher_entries(ids, scores)
    st, g = _dev32(row_stats(apart, 1.0)), _dev32(rng.normal(size=rows))
    targets = torch.from_numpy(ids[:, 2].astype(np.int32)).to(_dev())
    loss = torch.zeros(rows, device=_dev())
    out = Matrix(np.zeros((rows, V)), dtype, pad, start)
    for make in (lambda m, d: lg.LogProbsGrad(m.rows(), m.view, st, d, targets=targets,
                                              grad_logprob=g),
                 lambda m, d: lg.Distill(m.rows(), m.view, top, 9, lg.DISTILL_TAIL, loss,
                                         grad_loss=g, grad_logits=d)):
        make(apart, out.view).run()
        make(both, grad).run()
        torch.cuda.synchronize()
        assert torch.equal(grad, out.view) and torch.equal(both.view, apart.view)
        assert apart.outside_untouched() and out.outside_untouched()
        if gap:
            edges = torch.as_strided(both.flat, (rows - 1, gap), (both.stride, 1), both.stride - gap)
            assert (edges == both.marker).all()
            assert (torch.as_strided(both.flat, (rows, gap), (both.stride, 1), V) == both.marker).all()


def test_own_workspace_is_free_when_the_call_is_built(gpu_lib):
    """A call object built on one torch stream, over memory that stream still
    has writes queued for, and run on another: those writes come first."""
    import torch
    rng = np.random.default_rng(62)
    mat = Matrix(_logits(rng, 2, 60000), "bf16")
    r = mat.rows()
    want = run_logprobs(mat, 1.0, None, k=12)
    top = torch.zeros((2, 12, 2), dtype=torch.int32, device=_dev())
    big = torch.zeros(1 << 28, dtype=torch.float32, device=_dev())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        before = torch.zeros(lg.logprobs_workspace(r, 12), dtype=torch.uint8, device=_dev())
        for _ in range(20):
            big.add_(1.0)
        before.fill_(0xff)
        del before
        call = lg.LogProbs(r, mat.view, top_k=12, top=top)
    call.run()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(top.cpu().numpy(), want["top"])


def test_call_built_and_captured_in_one_graph(gpu_lib):
    """A call object with a workspace of its own, built while torch captures."""
    import torch
    mat = Matrix(_logits(np.random.default_rng(63), 2, 60000), "bf16")
    want = run_logprobs(mat, 1.0, None, k=12)
    top = torch.zeros((2, 12, 2), dtype=torch.int32, device=_dev())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call = lg.LogProbs(mat.rows(), mat.view, top_k=12, top=top)
        call.run(torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        top.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(top.cpu().numpy(), want["top"])


def test_workspace_contents_do_not_matter(gpu_lib):
    """A workspace filled with NaN patterns, larger than needed, and a call
    without one where one is needed."""
    import torch
    rng = np.random.default_rng(61)
    mat = Matrix(_logits(rng, 2, 50000), "bf16")
    r = mat.rows()
    need = lg.logprobs_workspace(r, 12)
    want = run_logprobs(mat, 1.0, None, k=12)
    top = torch.zeros((2, 12, 2), dtype=torch.int32, device=_dev())
    space = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=_dev())
    call = lg.LogProbs(r, mat.view, top_k=12, top=top, workspace=space)
    call.run()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(top.cpu().numpy(), want["top"])
    assert (space[need:] == 0xff).all()
    if need:
        small = lg.LogProbs(r, mat.view, top_k=12, top=top, workspace=space[:need - 16])
        assert small.submit() == ws.WS_E_INVALID_ARG
    ids, scores = make_teacher(rng, mat.z, 9, ol.TAIL)
    loss = torch.zeros(2, device=_dev())
    grad = torch.zeros((2, 50000), dtype=torch.bfloat16, device=_dev())
    need = lg.distill_workspace(r, lg.DISTILL_TAIL, True)
    space = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=_dev())
    lg.Distill(r, mat.view, teacher_entries(ids, scores), 9, lg.DISTILL_TAIL, loss,
               grad_loss=_dev32(np.ones(2)), grad_logits=grad, workspace=space).run()
    torch.cuda.synchronize()
    want, wgrad, _, _ = run_distill(mat, 1.0, ids, scores, ol.TAIL, np.ones(2))
    np.testing.assert_array_equal(loss.cpu().numpy(), want)
    np.testing.assert_array_equal(grad.double().cpu().numpy(), wgrad)
    assert (space[need:] == 0xff).all()


def test_two_threads_at_once(gpu_lib):
    """Two host threads, each with its own call objects and stream."""
    import threading

    import torch
    sets = [_all_calls(81, 2, 100001, "bf16"), _all_calls(82, 40, 5003, "f32")]
    alone = []
    for _, calls, outs in sets:
        for c in calls:
            c.run()
        torch.cuda.synchronize()
        alone.append(_bits(outs))
        for o in outs:
            o.zero_()
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    failed = []

    def work(calls, stream):
        try:
            for _ in range(50):
                for c in calls:
                    c.run(stream)
        except Exception as e:      # reported by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(calls, s.cuda_stream))
               for (_, calls, _), s in zip(sets, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for (_, _, outs), want in zip(sets, alone):
        for a, b in zip(_bits(outs), want):
            np.testing.assert_array_equal(a, b)


def test_calls_with_a_distillation_workspace_each(gpu_lib):
    """Loss and gradient in three kernels, whose statistics, tail and part sums
    lie in the workspace: two streams at once, a graph replayed, and a workspace
    of NaN patterns all give the bits of the calls alone."""
    import torch
    sets = [_all_calls(71, 2, 100001, "bf16"), _all_calls(72, 3, 90001, "f16")]
    for mat, _, _ in sets:
        assert lg.distill_workspace(mat.rows(1.1), lg.DISTILL_TAIL, True) > 0
    alone = []
    for _, calls, outs in sets:
        for c in calls:
            c.run()
        torch.cuda.synchronize()
        alone.append(_bits(outs))
    graphs = []
    for _, calls, _ in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for c in calls:
                c.run(torch.cuda.current_stream().cuda_stream)
    streams = [torch.cuda.Stream() for _ in sets]

    def clear():
        for _, calls, outs in sets:
            for o in outs:
                o.zero_()
            calls[-1]._keep[-1].fill_(0xff)
        torch.cuda.synchronize()

    def check():
        torch.cuda.synchronize()
        for (_, _, outs), want in zip(sets, alone):
            for a, b in zip(_bits(outs), want):
                np.testing.assert_array_equal(a, b)

    for _ in range(3):
        clear()
        for (_, calls, _), s in zip(sets, streams):
            for c in calls:
                c.run(s.cuda_stream)
        check()
        clear()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        check()


def test_refusals_on_the_device(gpu_lib):
    import torch
    z = torch.zeros((4, 100), device=_dev())
    ndev = torch.cuda.device_count()
    r = lg.make_rows(rows=4, vocab=100, device=ndev)
    assert lg.LogProbs(r, z.data_ptr()).submit() == ws.WS_E_NO_DEVICE
    r = lg.make_rows(rows=4, vocab=100)
    with pytest.raises(ValueError, match="strides"):
        lg.LogProbs(r, torch.zeros((4, 200), device=_dev())[:, ::2])
    with pytest.raises(ValueError, match="holds"):
        lg.LogProbs(r, z, entropy=torch.zeros(3, device=_dev()))
    with pytest.raises(ValueError, match="contiguous"):
        lg.LogProbs(r, z, entropy=torch.zeros(8, device=_dev())[::2])
    with pytest.raises(ValueError, match="shape"):
        lg.LogProbs(r, torch.zeros((4, 99), device=_dev()))
    stats = torch.zeros((4, 2), device=_dev())
    inside = z.flatten()[8:].data_ptr()
    assert lg.LogProbsGrad(r, z, stats, inside, grad_stride=100).submit() == ws.WS_E_INVALID_ARG
    torch.cuda.synchronize()
    assert (z == 0).all()
