"""Host half of the operators over rows of hidden states, on the CPU (no GPU,
no HIP launch): argument checks and launch geometry through the planning code
and through the built C ABI, ABI struct layouts, and the checks the Python
binding makes on tensors."""
import ctypes
import os
import subprocess
from ctypes import byref, c_size_t

import pytest
import torch

from post_processing_amd import build as ppbuild
from post_processing_amd import states as st
from post_processing_amd import ws


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("host") / "ws_states_test")
    return ppbuild.build_host_test(out, driver="ws_states_test")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(ws.LIB_PATH):
        ppbuild.build_lib()
    return st.load()


def _run(driver, *args, env=None):
    res = subprocess.run([driver, *args], capture_output=True, text=True, env=env)
    assert res.returncode == 0 and "runtime error" not in res.stderr, res.stdout + res.stderr
    return res.stdout


def test_selftest(driver):
    assert "\n0 failures" in "\n" + _run(driver, "selftest")


def test_selftest_under_sanitizers(tmp_path):
    out = ppbuild.build_host_test(str(tmp_path / "asan"), sanitize=True, driver="ws_states_test")
    assert "\n0 failures" in "\n" + _run(out, "selftest", env=dict(os.environ))


def test_abi_struct_layout(driver):
    mirrors = {"ws_states": st.States, "ws_norm_stats": st.NormStats,
               "ws_embed_args": st.EmbedArgs, "ws_embed_grad_args": st.EmbedGradArgs,
               "ws_layernorm_args": st.LayerNormArgs,
               "ws_layernorm_grad_args": st.LayerNormGradArgs}
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
    t = st.make_states(rows=4, width=100)
    n = c_size_t(7)
    assert lib.ws_embed(None, byref(st.EmbedArgs()), None) == ws.WS_E_INVALID_ARG
    assert lib.ws_embed(byref(t), None, None) == ws.WS_E_INVALID_ARG
    assert lib.ws_embed(byref(t), byref(st.EmbedArgs()), None) == ws.WS_E_INVALID_ARG
    assert lib.ws_embed_grad(byref(t), byref(st.EmbedGradArgs()), None) == ws.WS_E_INVALID_ARG
    assert lib.ws_layernorm(byref(t), byref(st.LayerNormArgs()), None) == ws.WS_E_INVALID_ARG
    assert lib.ws_layernorm_grad(byref(t), byref(st.LayerNormGradArgs()),
                                 None) == ws.WS_E_INVALID_ARG
    assert lib.ws_embed_grad_workspace(byref(t), 0, byref(n)) == ws.WS_E_INVALID_ARG
    assert lib.ws_embed_grad_workspace(byref(t), 10, None) == ws.WS_E_INVALID_ARG
    assert lib.ws_embed_grad_workspace(None, 10, byref(n)) == ws.WS_E_INVALID_ARG
    assert lib.ws_layernorm_grad_workspace(byref(t), None) == ws.WS_E_INVALID_ARG
    assert lib.ws_layernorm_grad_workspace(None, byref(n)) == ws.WS_E_INVALID_ARG
    assert n.value == 7


def test_no_rows_is_checked_and_does_nothing(lib):
    t = st.make_states(rows=0, width=100)
    a = st.EmbedArgs()
    assert lib.ws_embed(byref(t), byref(a), None) == ws.WS_E_INVALID_ARG     # vocab 0
    a.vocab, a.table_stride = 5, 100
    assert lib.ws_embed(byref(t), byref(a), None) == ws.WS_OK
    n = st.LayerNormArgs()
    n.y_stride = 100
    assert lib.ws_layernorm(byref(t), byref(n), None) == ws.WS_OK
    n.eps = -1.0
    assert lib.ws_layernorm(byref(t), byref(n), None) == ws.WS_E_INVALID_ARG
    g = st.EmbedGradArgs()
    g.vocab, g.grad_stride, g.accumulate, g.grad_table = 5, 100, 1, 4096
    assert lib.ws_embed_grad(byref(t), byref(g), None) == ws.WS_OK


def test_workspaces_are_checked(lib):
    t = st.make_states(rows=40, width=100)
    need = st.embed_grad_workspace(t, 1000)
    assert need >= 40 * 4 * 4 + 2 * 100 * 4
    for given, size in ((1 << 30, need - 1), ((1 << 30) + 8, need), (None, need)):
        call = st.EmbedGrad(t, 1 << 20, 1 << 21, 1 << 22, vocab=1000, workspace=1 << 30)
        call._args.workspace, call._args.workspace_bytes = given, size
        assert call.submit() == ws.WS_E_INVALID_ARG
    need = st.layernorm_grad_workspace(t)
    call = st.LayerNormGrad(t, 1 << 20, 1 << 21, 1 << 22, grad_weight=1 << 23, workspace=1 << 30)
    call._args.workspace_bytes = need - 1
    assert call.submit() == ws.WS_E_INVALID_ARG


def test_workspaces_over_other_buffers_are_refused(lib):
    """Few rows and many, through the built library: a workspace that begins in, or
    reaches into, what the call reads or writes."""
    for rows in (40, 5000):
        t = st.make_states(rows=rows, width=100)
        need = st.embed_grad_workspace(t, 1000)
        out, ids, table = 1 << 28, 1 << 27, 1 << 29
        for at in (out, out + 16, out - need + 16, ids, table, table - 16):
            call = st.EmbedGrad(t, out, ids, table, vocab=1000, workspace=at)
            assert call._args.workspace_bytes >= need
            assert call.submit() == ws.WS_E_INVALID_ARG, (rows, at)
        need = st.layernorm_grad_workspace(t)
        x, stats, gy, gx, weight, gw, gb = (i << 26 for i in range(1, 8))
        for at in (x, stats, gy, gx, gx - need + 16, weight, gw, gb):
            call = st.LayerNormGrad(t, x, stats, gy, grad_x=gx, weight=weight, grad_weight=gw,
                                    grad_bias=gb, workspace=at)
            assert call.submit() == ws.WS_E_INVALID_ARG, (rows, at)


def test_binding_checks_tensors(lib):
    """Type, device, size and layout of tensors are refused in Python, before an
    address is taken (CPU tensors stand for a wrong device)."""
    t = st.make_states(rows=4, width=100)
    x = torch.zeros(4, 100)
    meta = {"device": "meta"}
    with pytest.raises(ValueError, match="expected cuda:0"):
        st.LayerNorm(t, x, 4096)
    with pytest.raises(ValueError, match="torch.float64"):
        st.LayerNorm(t, x.double(), 4096)
    with pytest.raises(ValueError, match="int32"):
        st.Embed(t, 4096, torch.zeros(4, dtype=torch.int64, **meta), 8192, vocab=9)
    with pytest.raises(ValueError, match="float16"):
        st.LayerNorm(t, 4096, 8192, weight=torch.zeros(100, **meta), weight_dtype=ws.DTYPE_F16)
    with pytest.raises(ValueError, match="expected cuda:0"):
        st.EmbedGrad(t, 4096, 8192, torch.zeros(9, 100), vocab=9)
    with pytest.raises(ws.WsError):
        st.EmbedGrad(t, 4096, 8192, 1 << 20, vocab=0)


def test_sizes_and_strides_past_the_abi_are_refused_not_wrapped(lib):
    for bad in (dict(rows=2 ** 32 + 1), dict(width=2 ** 33), dict(dtype=2 ** 40)):
        with pytest.raises(ValueError, match="32"):
            st.make_states(**{**dict(rows=4, width=100), **bad})
    t = st.make_states(rows=4, width=100)
    with pytest.raises(ValueError, match="32"):
        st.Embed(t, 4096, 8192, 1 << 20, vocab=2 ** 32 + 5)
    for bad in (2 ** 64 + 100, 2 ** 63, -2 ** 64 + 100):
        with pytest.raises(ValueError, match="64 bits"):
            st.make_states(rows=4, width=100, row_stride=bad)
        with pytest.raises(ValueError, match="64 bits"):
            st.Embed(t, 4096, 8192, 1 << 20, vocab=5, table_stride=bad)
        with pytest.raises(ValueError, match="64 bits"):
            st.EmbedGrad(t, 4096, 8192, 1 << 20, vocab=5, grad_stride=bad)
        with pytest.raises(ValueError, match="64 bits"):
            st.LayerNorm(t, 4096, 1 << 20, y_stride=bad)
        with pytest.raises(ValueError, match="64 bits"):
            st.LayerNormGrad(t, 4096, 8192, 1 << 20, grad_x=1 << 21, grad_x_stride=bad)
