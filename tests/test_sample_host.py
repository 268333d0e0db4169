"""Host half of sampling, on the CPU (no GPU, no HIP launch): argument checks
and launch geometry through the planning code and the built C ABI, the ABI
struct's layout, the checks the Python binding makes, and what ties its oracle
to the definition."""
import ctypes
import os
import subprocess
from ctypes import byref, c_size_t

import numpy as np
import pytest
import torch

from oracle import logits as ol
from post_processing_amd import build as ppbuild
from post_processing_amd import logits as lg
from post_processing_amd import ws


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("host") / "ws_sample_test")
    return ppbuild.build_host_test(out, driver="ws_sample_test")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ws.LIB_PATH):
        ppbuild.build_lib()
    return lg.load()


def _run(driver, *args, env=None):
    res = subprocess.run([driver, *args], capture_output=True, text=True, env=env)
    assert res.returncode == 0 and "runtime error" not in res.stderr, res.stdout + res.stderr
    return res.stdout


def test_selftest(driver):
    assert "\n0 failures" in "\n" + _run(driver, "selftest")


def test_selftest_under_sanitizers(tmp_path):
    out = ppbuild.build_host_test(str(tmp_path / "asan"), sanitize=True, driver="ws_sample_test")
    assert "\n0 failures" in "\n" + _run(out, "selftest", env=dict(os.environ))


def test_abi_struct_layout(driver):
    seen = set()
    for line in _run(driver, "layout").splitlines():
        _, field, value = line.split()
        if field == "sizeof":
            assert ctypes.sizeof(lg.SampleArgs) == int(value)
        else:
            assert getattr(lg.SampleArgs, field).offset == int(value), field
            seen.add(field)
    assert seen == {f[0] for f in lg.SampleArgs._fields_}


def test_c_abi_refuses_before_it_touches_a_device(lib):
    r = lg.make_rows(rows=4, vocab=100)
    n = c_size_t(7)
    assert lib.ws_sample(None, byref(lg.SampleArgs()), None) == ws.WS_E_INVALID_ARG
    assert lib.ws_sample(byref(r), None, None) == ws.WS_E_INVALID_ARG
    assert lib.ws_sample(byref(r), byref(lg.SampleArgs()), None) == ws.WS_E_INVALID_ARG
    assert lib.ws_sample_workspace(None, byref(n)) == ws.WS_E_INVALID_ARG
    assert lib.ws_sample_workspace(byref(r), None) == ws.WS_E_INVALID_ARG
    assert n.value == 7
    none = lg.make_rows(rows=0, vocab=100)
    assert lib.ws_sample(byref(none), byref(lg.SampleArgs()), None) == ws.WS_OK


def test_outputs_over_other_buffers_are_refused(lib):
    """Through the built library, a workspace among them."""
    r = lg.make_rows(rows=4, vocab=100)
    assert lg.Sample(r, 1 << 20, 1 << 21, (1 << 20) + 400).submit() == ws.WS_E_INVALID_ARG
    assert lg.Sample(r, 1 << 20, 1 << 21, 1 << 21).submit() == ws.WS_E_INVALID_ARG
    assert lg.Sample(r, 1 << 20, 1 << 21, 1 << 22,
                     logprob=(1 << 22) + 12).submit() == ws.WS_E_INVALID_ARG
    one = lg.make_rows(rows=1, vocab=131072, dtype=ws.DTYPE_BF16)
    assert lg.sample_workspace(one) > 0
    for at in (1 << 20, (1 << 20) + 262144 - 16, 1 << 21, 1 << 22):
        call = lg.Sample(one, 1 << 20, 1 << 21, 1 << 22, workspace=at)
        assert call.submit() == ws.WS_E_INVALID_ARG, at


def test_binding_checks_tensors(lib):
    r = lg.make_rows(rows=4, vocab=100)
    meta = {"device": "meta"}
    with pytest.raises(ValueError, match="expected cuda:0"):
        lg.Sample(r, torch.zeros(4, 100), 4096, 4096)
    with pytest.raises(ValueError, match="float32"):
        lg.Sample(r, 4096, torch.zeros(4, dtype=torch.float64, **meta), 4096)
    with pytest.raises(ValueError, match="int32"):
        lg.Sample(r, 4096, 4096, torch.zeros(4, dtype=torch.int64, **meta))
    with pytest.raises(ValueError, match="int32"):
        lg.Sample(r, 4096, 4096, 4096, top_k=torch.zeros(4, **meta))
    call = lg.Sample(r, 4096, 4098, 4096)
    assert call.submit() == ws.WS_E_INVALID_ARG


# ---------------------------------------------------------------------------
# The oracle.


def test_oracle_keeps_what_the_definition_says():
    """Against the definition token by token, on few values so that ties are
    everywhere."""
    rng = np.random.default_rng(0)
    for _ in range(300):
        V = int(rng.integers(1, 12))
        z = rng.integers(-2, 3, V).astype(float)
        tau = float(rng.choice([0.5, 1.0, 2.0]))
        k, p = int(rng.integers(0, V + 2)), float(rng.choice([0.0, 0.37, 0.9, 1.0]))
        q = float(rng.choice([0.0, 0.2, 1.0]))
        before = [[j for j in range(V) if z[j] > z[i] or (z[j] == z[i] and j < i)] for i in range(V)]
        w = [np.exp((v - z.max()) / tau) for v in z]
        first = [i for i in range(V) if k == 0 or len(before[i]) < k]
        mass = sum(w[i] for i in first)
        want = [i for i in first
                if (p == 1 or not before[i] or sum(w[j] for j in before[i]) < p * mass - 1e-12)
                and w[i] >= q - 1e-12]
        kept, weights = ol.kept_tokens(z, tau, k, p, q)
        assert kept.tolist() == want, (z, tau, k, p, q)
        np.testing.assert_allclose(weights, [w[i] for i in want])


def test_oracle_draws_by_the_sum_up_to_a_token():
    z = np.log([1.0, 2.0, 4.0, 1.0])
    at = [ol.sample(z, u, 1.0)[0] for u in (0.0, 0.12, 0.13, 0.37, 0.38, 0.87, 0.88, 0.999)]
    assert at == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [ol.sample(z, u, 1.0, k=2)[0] for u in (0.0, 0.3, 0.34, 0.99)] == [1, 1, 2, 2]
    assert abs(ol.sample(z, 0.5, 1.0, k=2)[1] - np.log(4 / 6)) < 1e-15
    assert abs(ol.sample(z, 0.5, 0.5)[1] - np.log(16 / 22)) < 1e-15
    assert ol.sample(z, 0.1, 0.0) == (2, 0.0)


def test_oracle_rows_without_a_distribution():
    z = np.array([0.0, -np.inf, 1.0])
    assert ol.sample(z, 0.0, 1.0)[0] == 0
    for bad in (np.nan, np.inf):
        token, lp = ol.sample(np.array([0.0, bad, 1.0]), 0.5, 1.0)
        assert token == -1 and np.isnan(lp)
    assert ol.sample(np.full(3, -np.inf), 0.5, 1.0) == (-1, -np.inf)
    for given in (dict(u=1.0, tau=1.0), dict(u=0.5, tau=-1.0), dict(u=0.5, tau=1.0, k=-1),
                  dict(u=0.5, tau=1.0, p=1.5), dict(u=0.5, tau=1.0, q=-0.1)):
        assert ol.sample(z, **given)[0] == -1
