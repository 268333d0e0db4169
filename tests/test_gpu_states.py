"""The operators over rows of hidden states against the float64 oracle.

Tolerances, with E = 2^-24 the half step of FP32 and H that of the rows' type
(both relative), N the width:

* a sum over a row in FP32 adds at most E of its terms' sizes per addition on
  any element's way: at most ceil(N / 64) + 16 in a thread (a slot more than its
  share) and 16 to join lanes and waves, A(N) = ceil(N / 64) + 32 in all;
* mean: a first mean m0 off by s0 <= (A + 2) E mean|x|; the deviations from it,
  each rounded by E, are summed again, so the corrected mean is off by (A + 4) E
  mean|x - m0| and its own rounding;
* variance: (A + 5) E of the mean square about m0 (the variance and s0^2 at most)
  and of the square taken off; the inverse half of that over var + eps, relative,
  and 3 E for sum, root and division;
* y: the deviation's two differences, two products and a sum, each E of its
  result, and one rounding H;
* gradients: u = (x - mean) inverse is off by 3 E relative (the statistics are
  inputs), the row's two means by (A + 6) E of their terms' mean sizes, and each
  further operation by E of its result;
* sums over R rows, whatever their order: at most R additions on any way,
  (R + 4) E of the terms' sizes.
"""
import math

import numpy as np
import pytest

from oracle import states as os_
from post_processing_amd import states as st
from post_processing_amd import ws

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SMALLEST = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
CODE = {"f32": ws.DTYPE_F32, "f16": ws.DTYPE_F16, "bf16": ws.DTYPE_BF16}
TYPES = ["f32", "f16", "bf16"]
MARK = 7.0


def _type(dtype):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[dtype]


def _dev():
    import torch
    return torch.device("cuda:0")


class Matrix:
    """Rows on the GPU at a chosen offset and stride inside a larger buffer of a
    marker value, and their exact values in float64."""

    def __init__(self, values, dtype, pad=0, shift=0):
        import torch
        rows, width = values.shape
        self.stride, self.shift, self.shape, self.dtype = width + pad, shift, (rows, width), dtype
        self.flat = torch.full((shift + rows * self.stride + 16,), MARK, dtype=_type(dtype),
                               device=_dev())
        self.view = torch.as_strided(self.flat, (rows, width), (self.stride, 1), shift)
        if values.size:
            self.view.copy_(torch.from_numpy(np.array(values, order="C")).to(_dev()))
        self.v = self.get()

    def get(self):
        return self.view.double().cpu().numpy()

    def states(self):
        return st.make_states(rows=self.shape[0], width=self.shape[1], dtype=CODE[self.dtype],
                              row_stride=self.stride)

    def outside_untouched(self):
        import torch
        flat = self.flat.clone()
        torch.as_strided(flat, self.shape, (self.stride, 1), self.shift).fill_(MARK)
        return bool((flat == MARK).all())


def blank(rows, width, dtype, pad=0, shift=0):
    return Matrix(np.full((rows, width), -3.0), dtype, pad, shift)


def vector(values, dtype):
    import torch
    t = torch.from_numpy(np.asarray(values, dtype=np.float64)).to(_dev()).to(_type(dtype))
    return t, t.double().cpu().numpy()


def ids_on_gpu(ids):
    import torch
    return torch.from_numpy(np.asarray(ids, dtype=np.int32)).to(_dev())


def run(call, stream=None):
    import torch
    torch.cuda.synchronize()
    call.run(stream)
    torch.cuda.synchronize()


def assert_close(got, want, tol, what=""):
    got, want, tol = np.broadcast_arrays(np.asarray(got, dtype=np.float64), want, tol)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    fine = np.isfinite(want) & np.isfinite(got)
    assert (same | fine).all(), f"{what}: non-finite values differ"
    err = np.where(same | ~fine, 0.0, np.abs(np.where(fine, got, 0) - np.where(fine, want, 0)))
    over = err - np.where(same, np.inf, tol)
    if err.size:
        at = np.unravel_index(np.argmax(over), over.shape)
        assert (over <= 0).all(), f"{what}: error {err[at]:.3e} over {tol[at]:.3e} at {at}"


# ---------------------------------------------------------------------------
# Embedding lookup.


def check_embed(dtype, rows, width, vocab, scale=1.0, pad=0, shift=0, ids=None, seed=0):
    rng = np.random.default_rng(seed)
    table = Matrix(rng.normal(size=(vocab, width)), dtype, pad, shift)
    out = blank(rows, width, dtype, (pad * 3) % 7, (shift * 5) % 11)
    ids = rng.integers(-1, vocab, rows) if ids is None else np.asarray(ids)
    run(st.Embed(out.states(), table.view, ids_on_gpu(ids), out.view, vocab=vocab, scale=scale,
                 table_stride=table.stride))
    want = os_.embed(table.v, ids, float(np.float32(scale)))
    tol = np.abs(want) * (E + HALF[dtype] * (1 + E)) + SMALLEST[dtype]
    assert_close(out.get(), want, np.where(np.isnan(tol), 0, tol))
    assert out.outside_untouched() and table.outside_untouched()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [(1, 1), (1, 4096), (3, 7), (5, 8), (2, 9), (64, 64),
                                        (7, 1000), (33, 2049), (300, 65), (2, 9001)])
def test_embed_sizes(gpu_lib, dtype, rows, width):
    check_embed(dtype, rows, width, 50, scale=1.7, seed=rows * 7 + width)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 5), (0, 1), (8, 8), (7, 3)])
def test_embed_strides_and_starts(gpu_lib, dtype, pad, shift):
    check_embed(dtype, 19, 203, 31, scale=-0.3, pad=pad, shift=shift)


def test_embed_indices_outside(gpu_lib):
    check_embed("bf16", 9, 130, 11,
                ids=[-1, 0, 10, 11, -2, 2 ** 31 - 1, -2 ** 31, -1, 5])


def test_embed_scale_zero_and_infinities(gpu_lib):
    import torch
    table = torch.tensor([[1.0, float("inf"), float("nan"), -2.0]], device=_dev())
    out = torch.empty(1, 4, device=_dev())
    run(st.Embed(st.make_states(rows=1, width=4), table, ids_on_gpu([0]), out, vocab=1, scale=0.0))
    got = out.cpu().numpy()[0]
    assert got[0] == 0 and np.isnan(got[1]) and np.isnan(got[2]) and got[3] == 0


def test_embed_offsets_past_32_bits(gpu_lib):
    """A table of more than 2^32 elements, and rows written as far out."""
    import torch
    stride, vocab, width = (1 << 20) + 24, 4112, 40
    flat = torch.empty(vocab * stride, dtype=torch.bfloat16, device=_dev())
    table = torch.as_strided(flat, (vocab, width), (stride, 1))
    values = torch.arange(vocab * width, device=_dev()).view(vocab, width) % 251
    table.copy_(values)
    ids = torch.tensor([4111, 0, 4095, 4096], dtype=torch.int32, device=_dev())
    out = torch.empty(4, width, dtype=torch.bfloat16, device=_dev())
    shape = st.make_states(rows=4, width=width, dtype=ws.DTYPE_BF16)
    run(st.Embed(shape, table, ids, out, vocab=vocab, scale=1.0))
    assert torch.equal(out.long(), values[ids.long()])
    far = st.make_states(rows=vocab, width=width, dtype=ws.DTYPE_BF16, row_stride=stride)
    back = torch.arange(vocab - 1, -1, -1, dtype=torch.int32, device=_dev())
    packed = values.to(torch.bfloat16)
    run(st.Embed(far, packed, back, table, vocab=vocab, scale=1.0))
    assert torch.equal(table.long(), values.flip(0))


# ---------------------------------------------------------------------------
# Its gradient.


def check_embed_grad(dtype, ids, width, vocab, scale=1.0, grad_dtype=None, accumulate=False,
                     pad=0, shift=0, seed=0):
    rng = np.random.default_rng(seed)
    grad_dtype = grad_dtype or dtype
    ids = np.asarray(ids)
    grad = Matrix(rng.normal(size=(len(ids), width)), dtype, pad, shift)
    held = Matrix(rng.normal(size=(vocab, width)), grad_dtype, (pad * 3) % 7, (shift * 5) % 11)
    old = held.v
    run(st.EmbedGrad(grad.states(), grad.view, ids_on_gpu(ids), held.view, vocab=vocab,
                     grad_dtype=CODE[grad_dtype], grad_stride=held.stride, accumulate=accumulate,
                     scale=scale))
    scale = float(np.float32(scale))
    want = os_.embed_grad(grad.v, ids, vocab, scale, old if accumulate else None)
    size = os_.embed_grad(np.abs(grad.v), ids, vocab, abs(scale))
    count = os_.embed_grad(np.ones((len(ids), 1)), ids, vocab, 1.0)
    tol = (count + 2) * E * size + HALF[grad_dtype] * np.abs(want) * (1 + E) + SMALLEST[grad_dtype]
    tol += E * np.abs(want)
    got = held.get()
    assert_close(got, want, np.where(count > 0, tol, 0.0))
    assert held.outside_untouched() and grad.outside_untouched()
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 2, 31, 32, 33, 64, 65, 500, 2047, 2048, 2049, 5000])
def test_embed_grad_rows(gpu_lib, dtype, rows):
    rng = np.random.default_rng(rows)
    ids = np.minimum(rng.zipf(1.3, rows) - 1, 600)     # some outside the vocabulary
    check_embed_grad(dtype, ids, 40, 600, scale=1.7, seed=rows)


@pytest.mark.parametrize("width", [1, 3, 8, 9, 255, 2048, 2051, 5000])
def test_embed_grad_widths(gpu_lib, width):
    rng = np.random.default_rng(width)
    check_embed_grad("bf16", rng.integers(-1, 20, 150), width, 20, grad_dtype="f32")
    check_embed_grad("f32", rng.integers(-1, 20, 150), width, 20)


@pytest.mark.parametrize("vocab", [1, 2, 511, 512, 513, 262143, 262144, 300000])
def test_embed_grad_vocabularies(gpu_lib, vocab):
    """One, two and three digits of the sort, and the borders between them."""
    rng = np.random.default_rng(vocab)
    ids = rng.integers(-1, vocab, 3000)
    ids[:4] = [vocab - 1, 0, vocab, vocab - 1]
    check_embed_grad("f16", ids, 3, vocab)


@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 5), (0, 1), (8, 8), (7, 3)])
@pytest.mark.parametrize("dtype,grad_dtype", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_strides_and_accumulation(gpu_lib, pad, shift, dtype, grad_dtype, accumulate):
    rng = np.random.default_rng(pad)
    check_embed_grad(dtype, rng.integers(-1, 30, 203), 67, 30, scale=0.5, grad_dtype=grad_dtype,
                     accumulate=accumulate, pad=pad, shift=shift)


@pytest.mark.parametrize("ids", [[-1] * 40, [3] * 200, [3] * 32, [3] * 33, [2] * 31 + [3] * 34,
                                 [0] * 32 + [1] * 32 + [2] * 32, [5] + [4] * 4000 + [5],
                                 [-1, 7, -1, 7], [99, -5, 2 ** 31 - 1, -2 ** 31, 1]])
def test_embed_grad_runs(gpu_lib, ids):
    """Runs of one token that end on, in and behind a block of rows."""
    for accumulate in (False, True):
        check_embed_grad("f32", ids, 20, 8, accumulate=accumulate)


@pytest.mark.parametrize("dtype,grad_dtype", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows,width", [(1, 1), (5, 3), (64, 64), (65, 9), (130, 70), (640, 20), (200, 700),
                                        (100, 2100), (1023, 33), (1024, 260), (1025, 33)])
def test_embed_grad_few_rows(gpu_lib, dtype, grad_dtype, accumulate, rows, width):
    """One token of many rows, tokens of one, of some, and rows that name none."""
    rng = np.random.default_rng(rows + width)
    ids = rng.integers(-2, 50, rows)
    ids[rng.random(rows) < 0.3] = 17
    check_embed_grad(dtype, ids, width, 47, scale=1.3, grad_dtype=grad_dtype, accumulate=accumulate,
                     pad=rows % 3, seed=rows)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [(4000, 1), (3000, 9), (3000, 65), (2000, 130), (1500, 300),
                                        (1200, 700), (700, 2100)])
def test_embed_grad_long_runs(gpu_lib, dtype, rows, width):
    """Tokens that go on for many blocks of rows, from blocks side by side or apart."""
    rng = np.random.default_rng(rows)
    ids = np.sort(rng.integers(0, 30, rows))
    ids[rows // 8:] = np.where(np.arange(rows - rows // 8) < rows // 2, 31, 33)
    check_embed_grad(dtype, rng.permutation(ids), width, 40, scale=0.3, seed=width)


@pytest.mark.parametrize("rows,width,vocab", [(131072, 2, 700), (131073, 3, 5), (140000, 33, 50000),
                                              (300000, 8, 2)])
def test_embed_grad_many_tiles(gpu_lib, rows, width, vocab):
    rng = np.random.default_rng(rows)
    ids = rng.integers(-1, vocab, rows)
    ids[rng.random(rows) < 0.4] = vocab // 2
    check_embed_grad("bf16", ids, width, vocab, grad_dtype="f32")


def test_embed_grad_without_rows(gpu_lib):
    import torch
    held = torch.full((5, 6), 3.0, device=_dev())
    shape = st.make_states(rows=0, width=6)
    run(st.EmbedGrad(shape, None, None, held, vocab=5, accumulate=True))
    assert (held == 3).all()
    run(st.EmbedGrad(shape, None, None, held, vocab=5))
    assert (held == 0).all()


def test_embed_grad_order_of_equal_tokens_is_by_row(gpu_lib):
    """The same bits again and from another workspace: no sum hangs on timing."""
    import torch
    rng = np.random.default_rng(5)
    ids = ids_on_gpu(np.minimum(rng.zipf(1.2, 20000), 999))
    grad = torch.randn(20000, 200, device=_dev(), dtype=torch.bfloat16)
    shape = st.make_states(rows=20000, width=200, dtype=ws.DTYPE_BF16)
    first = None
    for _ in range(5):
        out = torch.empty(1000, 200, dtype=torch.float32, device=_dev())
        run(st.EmbedGrad(shape, grad, ids, out, vocab=1000, grad_dtype=ws.DTYPE_F32))
        first = out if first is None else first
        assert torch.equal(out, first)


def test_embed_grad_many_rows(gpu_lib):
    """More rows than blocks of the smallest size, most of one token."""
    import torch
    n, vocab, width = 300001, 1000, 8
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(-1, vocab, (n,), device=_dev(), generator=gen, dtype=torch.int32)
    ids[torch.rand(n, device=_dev(), generator=gen) < 0.6] = 77
    grad = torch.randn(n, width, device=_dev(), generator=gen)
    out = torch.empty(vocab, width, device=_dev())
    run(st.EmbedGrad(st.make_states(rows=n, width=width), grad, ids, out, vocab=vocab))
    want = os_.embed_grad(grad.cpu().numpy(), ids.cpu().numpy(), vocab, 1.0)
    size = os_.embed_grad(grad.abs().cpu().numpy(), ids.cpu().numpy(), vocab, 1.0)
    # 38 additions in a block and 8,192 between blocks at most, rounding errors of
    # either sign; counted in full all the same.
    assert_close(out.double().cpu().numpy(), want, (38 + 8192) * E * size)


# Past the few rows that go without a sort: which launches each of these sizes takes,
# and its block of sorted rows, is held by the host test of the launch rules.


@pytest.mark.parametrize("width", [1, 3, 8, 9, 255, 2048, 2051, 5000])
def test_embed_grad_sorted_widths(gpu_lib, width):
    rng = np.random.default_rng(width)
    check_embed_grad("bf16", rng.integers(-1, 20, 1025), width, 20, grad_dtype="f32")
    check_embed_grad("f32", rng.integers(-1, 400, 1025), width, 400)


@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 5), (0, 1), (8, 8), (7, 3)])
@pytest.mark.parametrize("dtype,grad_dtype", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows", [1100, 2100, 4500])
def test_embed_grad_sorted_strides_and_accumulation(gpu_lib, rows, pad, shift, dtype, grad_dtype,
                                                    accumulate):
    rng = np.random.default_rng(pad + rows)
    check_embed_grad(dtype, rng.integers(-1, 900, rows), 67, 900, scale=0.5, grad_dtype=grad_dtype,
                     accumulate=accumulate, pad=pad, shift=shift)


# (rows, width, type, rows of a block)
BLOCKS = [(1100, 20, "f32", 8), (3000, 20, "f32", 8), (5000, 20, "f32", 8), (1100, 300, "f32", 8),
          (5000, 300, "f16", 8), (2100, 2051, "f32", 12), (5000, 2051, "f32", 29),
          (16384, 2100, "bf16", 32)]


@pytest.mark.parametrize("rows,width,dtype,block", BLOCKS)
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_grad_sorted_runs(gpu_lib, rows, width, dtype, block, accumulate):
    """Runs of one token that end on a border of the blocks of sorted rows, a row before
    it and a row behind it, and go on for as many blocks as are joined at a time, one
    less and one more, and twice as many; a token of most rows, and rows that name none."""
    ends = [block, 2 * block, 4 * block]                      # on the border, one block or two
    ends += [5 * block - 1, 5 * block, 6 * block + 1, 7 * block]
    for blocks in (3, 15, 16, 17, 18, 33):                    # from a border to a border
        ends.append(ends[-1] + blocks * block)
    ends.append(ends[-1] + 16 * block + 1)                    # behind the border, and back on it
    ends.append(ends[-1] + 2 * block - 1)
    assert ends[-1] % block == 0 and ends[-1] < rows - 8
    counts = np.diff([0] + ends + [rows - 5])
    ids = np.repeat(2 * np.arange(len(counts)), counts)       # every other token has no row
    ids = np.concatenate([ids, [-1, 999, -1, 2 ** 31 - 1, -2 ** 31]])
    ids = np.random.default_rng(rows).permutation(ids)
    check_embed_grad(dtype, ids, width, 2 * len(counts) + 3, scale=0.7, accumulate=accumulate,
                     seed=width)


def test_embed_grad_blocks_past_the_most_workgroups(gpu_lib):
    """So many rows that the blocks grow past their usual size (33 rows here)."""
    import torch
    rows, width, vocab = 262200, 1032, 30
    gen = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.randint(-1, vocab, (rows,), device=_dev(), generator=gen, dtype=torch.int32)
    ids[torch.rand(rows, device=_dev(), generator=gen) < 0.4] = 7
    grad = torch.randn(rows, width, device=_dev(), generator=gen).bfloat16()
    out = torch.empty(vocab, width, device=_dev())
    shape = st.make_states(rows=rows, width=width, dtype=ws.DTYPE_BF16)
    run(st.EmbedGrad(shape, grad, ids, out, vocab=vocab, grad_dtype=ws.DTYPE_F32))
    named = ids >= 0
    at, exact = ids[named].long(), grad[named].double()
    sums = lambda v: torch.zeros(vocab, width, device=_dev(),  # noqa: E731
                                 dtype=torch.float64).index_add_(0, at, v)
    want = sums(exact).cpu().numpy()
    size = sums(exact.abs_()).cpu().numpy()
    count = torch.bincount(at, minlength=vocab)[:, None].cpu().numpy()
    # (float64's own sums are off by 2^-29 of this)
    assert_close(out.double().cpu().numpy(), want, (count + 2) * E * size + E * np.abs(want))


# ---------------------------------------------------------------------------
# Layer norm.


def _a(width):
    return math.ceil(width / 64) + 32


def norm_tolerances(x, weight, bias, eps, dtype):
    width = x.shape[1]
    A = _a(width)
    mean, inverse = os_.norm_stats(x, eps)
    a = np.abs(x - mean[:, None])
    var = (a * a).mean(1)
    s0 = (A + 2) * E * np.abs(x).mean(1)
    about = a.mean(1) + s0
    mean_tol = (A + 4) * E * about + 2 * E * np.abs(mean) + 1e-44
    var_tol = (A + 5) * E * (var + s0 ** 2) + (2 * A + 10) * E * s0 ** 2 + 1e-44
    inverse_rel = 0.5 * var_tol * inverse ** 2 + 3 * E
    g = np.ones(width) if weight is None else np.abs(weight)
    y = np.abs(os_.layernorm(x, weight, bias, eps))
    scale = inverse[:, None] * g
    y_tol = (scale * (2 * E * a + E * s0[:, None] + (A + 5) * E * about[:, None])
             + a * scale * (inverse_rel[:, None] + 3 * E) + 2 * E * y)
    return mean_tol, inverse_rel * inverse * 1.01, y_tol * 1.01 + HALF[dtype] * y + SMALLEST[dtype]


def check_norm(x, dtype, weight="f32", bias=True, eps=1e-5, pad=0, shift=0, in_place=False):
    rows, width = x.shape
    rng = np.random.default_rng(width)
    X = Matrix(x, dtype, pad, shift)
    Y = X if in_place else blank(rows, width, dtype, (pad * 3) % 7, (shift * 5) % 11)
    kind = weight or dtype
    w_dev, w = vector(rng.normal(size=width), kind) if weight else (None, None)
    b_dev, b = vector(rng.normal(size=width), kind) if bias else (None, None)
    import torch
    stats = torch.full((rows, 2), -5.0, device=_dev())
    run(st.LayerNorm(X.states(), X.view, Y.view, weight=w_dev, bias=b_dev,
                     weight_dtype=CODE[kind], eps=eps, stats=stats, y_stride=Y.stride))
    eps = float(np.float32(eps))
    mean, inverse = os_.norm_stats(X.v, eps)
    mean_tol, inverse_tol, y_tol = norm_tolerances(X.v, w, b, eps, dtype)
    got = stats.double().cpu().numpy()
    assert_close(got[:, 0], mean, mean_tol, "mean")
    assert_close(got[:, 1], inverse, inverse_tol, "inverse")
    assert_close(Y.get(), os_.layernorm(X.v, w, b, eps), y_tol, "y")
    assert Y.outside_untouched() and X.outside_untouched()


WIDTHS = [1, 2, 3, 7, 8, 9, 63, 64, 65, 255, 512, 513, 1000, 1023, 1024, 1025, 2048, 2049, 4096, 4100,
          8191, 8192, 8200, 16384, 16391, 32768, 32777, 70001]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_widths(gpu_lib, dtype, width):
    rng = np.random.default_rng(width)
    check_norm(rng.normal(size=(5, width)) * 3 + 1, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 2, 3, 63, 1000, 5000])
def test_norm_rows(gpu_lib, dtype, rows):
    rng = np.random.default_rng(rows)
    check_norm(rng.normal(size=(rows, 129)), dtype, weight=dtype)


NARROW = [(1, 8), (3, 16), (7, 31), (8, 64), (9, 33), (15, 9), (17, 64), (2, 65), (3, 128), (4, 129),
          (5, 256), (31, 200), (1001, 40), (40000, 33), (20000, 130)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", NARROW)
def test_norm_narrow_rows(gpu_lib, dtype, rows, width):
    rng = np.random.default_rng(rows + width)
    check_norm(rng.normal(size=(rows, width)) * 2 - 1, dtype, weight=dtype, pad=rows % 4)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 5), (0, 1), (8, 8), (7, 3)])
@pytest.mark.parametrize("width", [5, 203, 2050])
def test_norm_strides_and_starts(gpu_lib, dtype, pad, shift, width):
    rng = np.random.default_rng(width)
    check_norm(rng.normal(size=(7, width)), dtype, weight=dtype, pad=pad, shift=shift)


@pytest.mark.parametrize("weight", [None, "f32", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("width", [100, 3001])
def test_norm_weights(gpu_lib, weight, bias, width):
    rng = np.random.default_rng(3)
    check_norm(rng.normal(size=(4, width)), "bf16", weight=weight, bias=bias)


@pytest.mark.parametrize("width", [60, 1001, 40000])
def test_norm_in_place(gpu_lib, width):
    rng = np.random.default_rng(4)
    check_norm(rng.normal(size=(9, width)), "f16", in_place=True, pad=2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [30, 900, 40000])
def test_norm_rows_far_from_zero(gpu_lib, dtype, width):
    """Offsets of thousands of deviations, constant rows, tiny and huge rows."""
    rng = np.random.default_rng(6)
    z = rng.normal(size=(8, width))
    top = 200.0 if dtype == "f16" else 1e15
    rows = [z[0] + 1000, z[1] * 0.1 - 5000, np.full(width, 1000.125), np.full(width, -3.0),
            np.zeros(width), z[2] * 1e-6, z[3] * top, np.where(np.arange(width) == 3, 5e4, z[4])]
    for eps in (1e-5, 1e-12):
        check_norm(np.stack(rows), dtype, eps=eps)


def test_norm_keeps_nan_and_infinity_in_their_rows(gpu_lib):
    import torch
    for width in (50, 1500, 40000):
        x = torch.randn(4, width, device=_dev())
        x[1, 3] = float("nan")
        x[2, 7] = float("inf")
        clean = x[[0, 3]].clone()
        y, y2 = torch.empty_like(x), torch.empty_like(clean)
        run(st.LayerNorm(st.make_states(rows=4, width=width), x, y))
        run(st.LayerNorm(st.make_states(rows=2, width=width), clean, y2))
        assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
        assert torch.equal(y[[0, 3]], y2)


def _rows_with_nan_and_infinity(width, seed=9):
    """Clean rows among ones that hold a NaN, an infinity of either sign, and both."""
    x = np.random.default_rng(seed).normal(size=(7, width))
    x[1, width // 2] = np.nan
    x[2, width - 1] = np.inf
    x[3, 0] = -np.inf
    x[5, 0], x[5, width - 1] = np.inf, -np.inf
    return x


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [3, 8, 50, 600, 1500, 8200, 16384, 40000, 70001])
def test_norm_statistics_of_nan_and_infinity(gpu_lib, dtype, width):
    """The statistics are the formulas' as well: a deviation of NaN, and a mean that is
    the infinity where the row's infinities have one sign."""
    x = _rows_with_nan_and_infinity(width)
    with np.errstate(invalid="ignore"):
        mean, inverse = os_.norm_stats(x, 1e-5)
        assert np.isnan(inverse[[1, 2, 3, 5]]).all() and np.isfinite(inverse[[0, 4, 6]]).all()
        assert mean[2] == np.inf and mean[3] == -np.inf and np.isnan(mean[[1, 5]]).all()
        check_norm(x, dtype, weight=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [4, 50, 1500, 40000])
def test_norm_of_sums_past_the_range(gpu_lib, dtype, width):
    """A sum that overflows makes its row NaN, squares that do an inverse of 0; the rows
    between them are as they are alone."""
    import torch
    x = torch.from_numpy(np.random.default_rng(2).normal(size=(4, width))).to(_dev()).to(_type(dtype))
    x[1] = 3e38
    x[3] = 0.0
    x[3, 0], x[3, 1] = 1e25, -1e25                 # a mean of 0, squares of 1e50
    y, stats = torch.empty_like(x), torch.empty(4, 2, device=_dev())
    run(st.LayerNorm(st.make_states(rows=4, width=width, dtype=CODE[dtype]), x, y, stats=stats))
    assert torch.isnan(y[1]).all() and torch.isnan(stats[1, 1])
    assert stats[3, 1] == 0 and (y[3] == 0).all()
    clean, alone = x[[0, 2]].contiguous(), torch.empty(2, width, device=_dev(), dtype=x.dtype)
    run(st.LayerNorm(st.make_states(rows=2, width=width, dtype=CODE[dtype]), clean, alone))
    assert torch.equal(y[[0, 2]], alone) and torch.isfinite(stats[[0, 2]]).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", [3, 50, 1500, 40000])
def test_norm_grad_of_nan_and_infinity(gpu_lib, dtype, width):
    """A forward's statistics of such rows: their gradients are NaN, the other rows'
    those of a call without them, the weight's NaN and the bias's finite."""
    import torch
    x = torch.from_numpy(_rows_with_nan_and_infinity(width)).to(_dev()).to(_type(dtype))
    g = torch.from_numpy(np.random.default_rng(1).normal(size=(7, width))).to(_dev()).to(_type(dtype))
    clean = [0, 4, 6]

    def step(x, g):
        rows = x.shape[0]
        shape = st.make_states(rows=rows, width=width, dtype=CODE[dtype])
        y, gx = torch.empty_like(x), torch.empty_like(x)
        stats = torch.empty(rows, 2, device=_dev())
        gw, gb = torch.empty(width, device=_dev()), torch.empty(width, device=_dev())
        run(st.LayerNorm(shape, x, y, stats=stats))
        run(st.LayerNormGrad(shape, x, stats, g, weight_dtype=ws.DTYPE_F32, grad_x=gx, grad_weight=gw,
                             grad_bias=gb))
        return gx, gw, gb

    gx, gw, gb = step(x, g)
    want, _, _ = step(x[clean].contiguous(), g[clean].contiguous())
    assert torch.equal(gx[clean], want)
    assert torch.isnan(gx[[1, 2, 3, 5]]).all()
    assert torch.isnan(gw).all() and torch.isfinite(gb).all()


def check_norm_grad(x, grad, dtype, weight="f32", pad=0, shift=0, in_place=None, eps=1e-5,
                    parts=("grad_x", "grad_weight", "grad_bias")):
    import torch
    rows, width = x.shape
    rng = np.random.default_rng(width + 1)
    X, G = Matrix(x, dtype, pad, shift), Matrix(grad, dtype, (pad * 5) % 9, (shift * 3) % 13)
    kind = weight or dtype
    w_dev, w = vector(rng.normal(size=width), kind) if weight else (None, None)
    mean, inverse = os_.norm_stats(X.v, eps)
    stats = torch.from_numpy(np.stack([mean, inverse], 1)).float().to(_dev())
    mean, inverse = stats.double().cpu().numpy().T
    O = {"x": X, "y": G}.get(in_place) or blank(rows, width, dtype, (pad * 3) % 7, (shift * 5) % 11)
    gw = torch.full((width,), -5.0, device=_dev(), dtype=_type(kind))
    gb = torch.full((width,), -5.0, device=_dev(), dtype=_type(kind))
    outs = {"grad_x": O.view, "grad_weight": gw, "grad_bias": gb}
    more = {"grad_x_stride": O.stride} if "grad_x" in parts else {}
    run(st.LayerNormGrad(X.states(), X.view, stats, G.view, weight=w_dev, weight_dtype=CODE[kind],
                         grad_y_stride=G.stride, **{k: outs[k] for k in parts}, **more))
    want = os_.layernorm_grad(X.v, mean, inverse, w, G.v)
    A = _a(width)
    u = np.abs((X.v - mean[:, None]) * inverse[:, None])
    d = np.abs(G.v) * (1 if w is None else np.abs(w))
    level = d.mean(1, keepdims=True)
    along = (d * u).mean(1, keepdims=True)
    dx = np.abs(want[0])
    tol = inverse[:, None] * (3 * E * d + (A + 8) * E * level + u * (A + 12) * E * along) + 3 * E * dx
    if "grad_x" in parts:
        assert_close(O.get(), want[0], tol * 1.01 + HALF[dtype] * dx + SMALLEST[dtype], "grad_x")
    for key, full, size in (("grad_weight", want[1], np.abs(G.v) * u),
                            ("grad_bias", want[2], np.abs(G.v))):
        if key in parts:
            tol = (rows + 4) * E * size.sum(0) * 1.01 + HALF[kind] * np.abs(full) + SMALLEST[kind]
            assert_close(outs[key].double().cpu().numpy(), full, tol, key)
    assert O.outside_untouched() and X.outside_untouched() and G.outside_untouched()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_grad_widths(gpu_lib, dtype, width):
    rng = np.random.default_rng(width)
    check_norm_grad(rng.normal(size=(5, width)) * 3 + 1, rng.normal(size=(5, width)), dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 63, 1000, 5001])
def test_norm_grad_rows(gpu_lib, dtype, rows):
    rng = np.random.default_rng(rows)
    check_norm_grad(rng.normal(size=(rows, 129)), rng.normal(size=(rows, 129)), dtype, weight=dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", NARROW)
def test_norm_grad_narrow_rows(gpu_lib, dtype, rows, width):
    rng = np.random.default_rng(rows + width)
    check_norm_grad(rng.normal(size=(rows, width)) * 2 - 1, rng.normal(size=(rows, width)), dtype,
                    weight=dtype, pad=rows % 4)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(1, 0), (3, 5), (0, 1), (8, 8), (7, 3)])
@pytest.mark.parametrize("width", [5, 203, 2050])
def test_norm_grad_strides_and_starts(gpu_lib, dtype, pad, shift, width):
    rng = np.random.default_rng(width)
    check_norm_grad(rng.normal(size=(7, width)), rng.normal(size=(7, width)), dtype, weight=dtype,
                    pad=pad, shift=shift)


@pytest.mark.parametrize("weight", [None, "f32", "bf16"])
@pytest.mark.parametrize("parts", [("grad_x",), ("grad_weight",), ("grad_bias",),
                                   ("grad_weight", "grad_bias"), ("grad_x", "grad_bias")])
@pytest.mark.parametrize("width", [100, 3001, 40000])
def test_norm_grad_parts(gpu_lib, weight, parts, width):
    rng = np.random.default_rng(3)
    check_norm_grad(rng.normal(size=(20, width)), rng.normal(size=(20, width)), "bf16",
                    weight=weight, parts=parts)


@pytest.mark.parametrize("in_place", ["x", "y"])
@pytest.mark.parametrize("width", [60, 1001, 40000])
def test_norm_grad_in_place(gpu_lib, in_place, width):
    rng = np.random.default_rng(4)
    check_norm_grad(rng.normal(size=(300, width)), rng.normal(size=(300, width)), "f16",
                    in_place=in_place)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [(3, 1500), (3, 6001), (3, 10300), (2, 12288), (2, 14000), (2, 20000),
                                        (2, 24600), (1500, 1100), (1100, 4200), (600, 8203), (300, 10300)])
def test_norm_threads_and_slots(gpu_lib, dtype, rows, width):
    """Rows of every number of slots a thread, and more rows than workgroups."""
    rng = np.random.default_rng(rows + width)
    x, grad = rng.normal(size=(2, rows, width))
    check_norm(x + 0.5, dtype, weight=dtype)
    check_norm_grad(x + 0.5, grad, dtype, weight=dtype)


def test_norm_more_rows_than_workgroups(gpu_lib):
    """Rows of less than a slot, some of which share a workgroup."""
    rng = np.random.default_rng(1)
    x, grad = rng.normal(size=(2, (1 << 20) + 3, 3))
    check_norm(x, "bf16", weight="bf16")
    check_norm_grad(x, grad, "bf16", weight="bf16")


def test_norm_grad_without_rows(gpu_lib):
    import torch
    gw, gb = torch.full((70,), 3.0, device=_dev()), torch.full((70,), 3.0, device=_dev())
    run(st.LayerNormGrad(st.make_states(rows=0, width=70), None, None, None, grad_weight=gw,
                         grad_bias=gb))
    assert (gw == 0).all() and (gb == 0).all()


# ---------------------------------------------------------------------------
# Streams, graphs, calls at once.


def _many_calls(seed, rows=700, width=520, vocab=900):
    """Every operator on its own buffers: calls, and the tensors they write."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    f = lambda *s: torch.randn(*s, device=_dev(), generator=gen).bfloat16()  # noqa: E731
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, device=_dev(), dtype=dtype)  # noqa: E731
    shape = st.make_states(rows=rows, width=width, dtype=ws.DTYPE_BF16)
    ids = torch.randint(-1, vocab, (rows,), device=_dev(), generator=gen, dtype=torch.int32)
    table, weight, bias, gy = f(vocab, width), f(width), f(width), f(rows, width)
    x, y, gx = e(rows, width), e(rows, width), e(rows, width)
    stats, gw, gb, gt = e(rows, 2, dtype=torch.float32), e(width), e(width), e(vocab, width)
    calls = [st.Embed(shape, table, ids, x, vocab=vocab, scale=3.0),
             st.LayerNorm(shape, x, y, weight=weight, bias=bias, stats=stats),
             st.LayerNormGrad(shape, x, stats, gy, weight=weight, grad_x=gx, grad_weight=gw,
                              grad_bias=gb),
             st.EmbedGrad(shape, gx, ids, gt, vocab=vocab, scale=3.0)]
    return calls, [x, y, stats, gx, gw, gb, gt], (table, ids, gy)


def _run_all(calls, stream):
    for c in calls:
        c.run(stream)


def test_states_on_two_streams_at_once(gpu_lib):
    import torch
    sets = [_many_calls(s) for s in (1, 2)]
    torch.cuda.synchronize()
    for calls, outs, _ in sets:
        _run_all(calls, None)
    torch.cuda.synchronize()
    want = [[o.clone() for o in outs] for _, outs, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for outs in (outs for _, outs, _ in sets):
        for o in outs:
            o.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(20):
        for (calls, _, _), s in zip(sets, streams):
            _run_all(calls, s.cuda_stream)
    torch.cuda.synchronize()
    for (_, outs, _), w in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))


def test_states_captured_and_replayed(gpu_lib):
    """A whole step captured once and replayed on new inputs, with eager work
    between the replays."""
    import torch
    calls, outs, (table, ids, gy) = _many_calls(3)
    twin, twin_outs, (table2, ids2, gy2) = _many_calls(3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run_all(calls, torch.cuda.current_stream().cuda_stream)
    for k in range(4):
        gen = torch.Generator(device="cuda").manual_seed(10 + k)
        table.copy_(torch.randn(table.shape, device=_dev(), generator=gen))
        gy.copy_(torch.randn(gy.shape, device=_dev(), generator=gen))
        ids.copy_(torch.randint(-1, 900, ids.shape, device=_dev(), generator=gen))
        for a, b in ((table2, table), (gy2, gy), (ids2, ids)):
            a.copy_(b)
        for o in outs + twin_outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        _run_all(twin, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, twin_outs)), k


# Gradients of the lookup that take a sort: in one workgroup's LDS, by two tiles that
# count for themselves, by three that are counted first, and by more than the tiles that
# add the counts themselves.
SORTED = [(1500, 520, 900), (2100, 520, 900), (5000, 520, 900), (140000, 40, 900)]


@pytest.mark.parametrize("rows,width,vocab", SORTED)
def test_sorted_states_on_two_streams_at_once(gpu_lib, rows, width, vocab):
    import torch
    sets = [_many_calls(s, rows, width, vocab) for s in (1, 2)]
    torch.cuda.synchronize()
    for calls, _, _ in sets:
        _run_all(calls, None)
    torch.cuda.synchronize()
    want = [[o.clone() for o in outs] for _, outs, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for _, outs, _ in sets:
        for o in outs:
            o.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(20):
        for (calls, _, _), s in zip(sets, streams):
            _run_all(calls, s.cuda_stream)
    torch.cuda.synchronize()
    for (_, outs, _), w in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(outs, w))


@pytest.mark.parametrize("rows,width,vocab", SORTED)
def test_sorted_states_captured_and_replayed(gpu_lib, rows, width, vocab):
    import torch
    calls, outs, (table, ids, gy) = _many_calls(3, rows, width, vocab)
    twin, twin_outs, (table2, ids2, gy2) = _many_calls(3, rows, width, vocab)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run_all(calls, torch.cuda.current_stream().cuda_stream)
    for k in range(4):
        gen = torch.Generator(device="cuda").manual_seed(10 + k)
        table.copy_(torch.randn(table.shape, device=_dev(), generator=gen))
        gy.copy_(torch.randn(gy.shape, device=_dev(), generator=gen))
        ids.copy_(torch.randint(-1, vocab, ids.shape, device=_dev(), generator=gen))
        if k == 2:
            ids[: rows // 2] = 5                              # one token of half the rows
        for a, b in ((table2, table), (gy2, gy), (ids2, ids)):
            a.copy_(b)
        for o in outs + twin_outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        _run_all(twin, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, twin_outs)), k
        want = os_.embed_grad(outs[3].double().cpu().numpy(), ids.cpu().numpy(), vocab, 3.0)
        size = os_.embed_grad(outs[3].double().abs().cpu().numpy(), ids.cpu().numpy(), vocab, 3.0)
        count = torch.bincount(ids[ids >= 0].long(), minlength=vocab)[:, None].cpu().numpy()
        tol = (count + 3) * E * size + HALF["bf16"] * np.abs(want) * (1 + E) + SMALLEST["bf16"]
        assert_close(outs[-1].double().cpu().numpy(), want, np.where(count > 0, tol, 0.0))


def test_states_refuse_another_device(gpu_lib):
    import torch
    shape = st.make_states(rows=1, width=4, device=torch.cuda.device_count())
    call = st.LayerNorm(shape, 4096, 8192)
    assert call.submit() == ws.WS_E_NO_DEVICE
