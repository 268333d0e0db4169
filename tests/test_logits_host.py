"""Host half of the operators over rows of logits, on the CPU (no GPU, no HIP
launch): argument checks through the planning code and through the built C
ABI, ABI struct layouts, and the checks the Python binding makes on tensors."""
import ctypes
import os
import subprocess
from ctypes import byref, c_size_t

import pytest
import torch

from post_processing_amd import build as ppbuild
from post_processing_amd import logits as lg
from post_processing_amd import ws


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("host") / "ws_logits_test")
    return ppbuild.build_host_test(out, driver="ws_logits_test")


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
    assert "0 failures" in _run(driver, "selftest")


def test_selftest_under_sanitizers(tmp_path):
    out = ppbuild.build_host_test(str(tmp_path / "asan"), sanitize=True, driver="ws_logits_test")
    assert "0 failures" in _run(out, "selftest", env=dict(os.environ))


def test_abi_struct_layout(driver):
    mirrors = {"ws_rows": lg.Rows, "ws_row_stats": lg.RowStats,
               "ws_logprobs_args": lg.LogProbsArgs,
               "ws_logprobs_grad_args": lg.LogProbsGradArgs, "ws_distill_args": lg.DistillArgs,
               "ws_distill_grad_args": lg.DistillGradArgs}
    seen = {name: set() for name in mirrors}
    for line in _run(driver, "layout").splitlines():
        struct, field, value = line.split()
        if field == "sizeof":
            assert ctypes.sizeof(mirrors[struct]) == int(value), struct
        else:
            assert getattr(mirrors[struct], field).offset == int(value), (struct, field)
            seen[struct].add(field)
    for name, mirror in mirrors.items():
        assert seen[name] == {f[0] for f in mirror._fields_}, name


def test_c_abi_refuses_before_it_touches_a_device(lib):
    """Every refusal the host can decide comes back without a GPU present."""
    r = lg.make_rows(rows=4, vocab=100)
    n = c_size_t(7)
    assert lib.ws_logprobs(None, byref(lg.LogProbsArgs()), None) == ws.WS_E_INVALID_ARG
    assert lib.ws_logprobs(byref(r), None, None) == ws.WS_E_INVALID_ARG
    assert lib.ws_logprobs(byref(r), byref(lg.LogProbsArgs()), None) == ws.WS_E_INVALID_ARG
    assert lib.ws_logprobs_grad(byref(r), byref(lg.LogProbsGradArgs()),
                                None) == ws.WS_E_INVALID_ARG
    assert lib.ws_distill(byref(r), byref(lg.DistillArgs()), None) == ws.WS_E_INVALID_ARG
    assert lib.ws_distill_grad(byref(r), byref(lg.DistillGradArgs()),
                               None) == ws.WS_E_INVALID_ARG
    assert lib.ws_logprobs_workspace(byref(r), 33, byref(n)) == ws.WS_E_INVALID_ARG
    assert lib.ws_logprobs_workspace(byref(r), 5, None) == ws.WS_E_INVALID_ARG
    assert lib.ws_distill_workspace(byref(r), 2, 0, byref(n)) == ws.WS_E_INVALID_ARG
    assert lib.ws_distill_workspace(byref(r), 1, 2, byref(n)) == ws.WS_E_INVALID_ARG
    assert lib.ws_distill_workspace(byref(r), 1, 1, None) == ws.WS_E_INVALID_ARG
    assert n.value == 7


def test_no_rows_is_checked_and_does_nothing(lib):
    r = lg.make_rows(rows=0, vocab=100)
    a = lg.LogProbsArgs()
    assert lib.ws_logprobs(byref(r), byref(a), None) == ws.WS_OK
    a.top_k = 33
    assert lib.ws_logprobs(byref(r), byref(a), None) == ws.WS_E_INVALID_ARG
    d = lg.DistillArgs()
    assert lib.ws_distill(byref(r), byref(d), None) == ws.WS_E_INVALID_ARG      # teacher_k 0
    d.teacher_k = 4
    assert lib.ws_distill(byref(r), byref(d), None) == ws.WS_OK
    g = lg.LogProbsGradArgs()
    g.grad_stride = 100
    assert lib.ws_logprobs_grad(byref(r), byref(g), None) == ws.WS_OK
    dg = lg.DistillGradArgs()
    dg.teacher_k = 4
    dg.grad_stride = 100
    assert lib.ws_distill_grad(byref(r), byref(dg), None) == ws.WS_OK


def test_binding_checks_tensors(lib):
    """Type, device, size and layout of tensors are refused in Python, before
    an address is taken (CPU tensors stand for a wrong device)."""
    r = lg.make_rows(rows=4, vocab=100)
    z = torch.zeros(4, 100)
    with pytest.raises(ValueError, match="expected cuda:0"):
        lg.LogProbs(r, z)
    with pytest.raises(ValueError, match="torch.float64"):
        lg.LogProbs(r, z.double())
    meta = {"device": "meta"}
    with pytest.raises(ValueError, match="expected cuda:0"):
        lg.Distill(r, 4096, torch.zeros(4, 8, 2, dtype=torch.int32, **meta), 8, lg.DISTILL_TAIL,
                   4096)
    with pytest.raises(ValueError, match="int32"):
        lg.LogProbs(r, 4096, targets=torch.zeros(4, dtype=torch.int64, **meta), logprob=4096)
    with pytest.raises(ws.WsError):
        lg.LogProbs(r, 4096, top_k=33, top=4096)
    with pytest.raises(ws.WsError):
        lg.Distill(r, 4096, 4096, 4, 5, 4096)


def test_bound_call_refuses_bad_addresses(lib):
    r = lg.make_rows(rows=4, vocab=100)
    call = lg.LogProbs(r, 4097)                   # not element aligned
    assert call.submit() == ws.WS_E_INVALID_ARG
    with pytest.raises(ws.WsError):
        call.run()


def test_sizes_past_the_abi_are_refused_not_wrapped(lib):
    for bad in (dict(rows=2 ** 32 + 1), dict(vocab=2 ** 33), dict(dtype=2 ** 40)):
        with pytest.raises(ValueError, match="32"):
            lg.make_rows(**{**dict(rows=4, vocab=100), **bad})
    with pytest.raises(ValueError, match="32"):
        lg.LogProbs(lg.make_rows(rows=4, vocab=100), 4096, top_k=2 ** 32)
    with pytest.raises(ValueError, match="32"):
        lg.Distill(lg.make_rows(rows=4, vocab=100), 4096, 4096, 2 ** 32 + 4, 0, 4096)


def test_workspace_tensor_is_checked(lib):
    with pytest.raises(ValueError, match="workspace"):
        lg.LogProbs(lg.make_rows(rows=1, vocab=131072, dtype=ws.DTYPE_BF16), 4096,
                    workspace=torch.zeros(1 << 20, dtype=torch.uint8))


@pytest.mark.parametrize("capturing", [False, True])
def test_own_workspace_is_free_before_any_stream_may_use_it(lib, monkeypatch, capturing):
    """torch's memory is free in the order of its current stream only, and a run
    may go to any stream: building waits for that stream (unless it is being
    captured, where waiting is an error)."""
    done = []

    class Stream:
        def synchronize(self):
            done.append("wait")

    def empty(*size, **kw):
        done.append("memory")
        return torch.zeros(*size, dtype=kw["dtype"])

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    lg.LogProbs(lg.make_rows(rows=1, vocab=131072, dtype=ws.DTYPE_BF16), 4096)
    assert done == (["memory"] if capturing else ["memory", "wait"])
    done.clear()
    lg.LogProbs(lg.make_rows(rows=1, vocab=100), 4096)          # needs none
    assert done == []


def test_strides_past_the_abi_are_refused_not_wrapped(lib):
    """2^64 + 100 is no stride of 100."""
    for bad in (2 ** 64 + 100, 2 ** 63, -2 ** 64 + 100):
        with pytest.raises(ValueError, match="64 bits"):
            lg.make_rows(rows=4, vocab=100, row_stride=bad)
        r = lg.make_rows(rows=4, vocab=100)
        with pytest.raises(ValueError, match="64 bits"):
            lg.LogProbsGrad(r, 4096, 4096, 1 << 20, grad_stride=bad)
        with pytest.raises(ValueError, match="64 bits"):
            lg.Distill(r, 4096, 4096, 4, lg.DISTILL_TAIL, 4096, grad_loss=4096,
                       grad_logits=1 << 20, grad_stride=bad)
        with pytest.raises(ValueError, match="64 bits"):
            lg.DistillGrad(r, 4096, 4096, 4, lg.DISTILL_RENORM, 4096, 4096, 1 << 20,
                           grad_stride=bad)
