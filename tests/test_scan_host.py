"""Refusals of the gated-scan and residual-norm entry points, through the C ABI and the
Python binding.  They return before any HIP call, so they run without a GPU; the host code
also runs under address and undefined-behaviour sanitizers with stub launchers
(tests/sanitize/scan_driver.cpp)."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import gated_delta_rule_short_amd as kda
from gated_delta_rule_short_amd import kda as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"
INV, UNS = K.KDA_ERR_INVALID_ARG, K.KDA_ERR_UNSUPPORTED
BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        from gated_delta_rule_short_amd import _build
        _build.build()
    return K.load_library()


def _addr(i):
    return 0x100000000 * (i + 1)


def _fill(a, names, kw):
    for i, f in enumerate(names):
        setattr(a, f, _addr(i))
    for f, v in kw.items():
        setattr(a, f, v)
    return a


def _scan(**kw):
    return _fill(K.KdaGatedScanArgs(num_seqs=2, channels=72, total_tokens=64, dtype=K.KDA_BF16),
                 ("x", "gate", "state_in", "state_out", "o", "cu_seqlens"), kw)


def _step(**kw):
    return _fill(K.KdaGatedScanDecodeArgs(num_seqs=2, channels=72, dtype=K.KDA_BF16), ("x", "gate", "state", "o"), kw)


def _grad(**kw):
    return _fill(K.KdaGatedScanBackwardArgs(num_seqs=2, channels=72, total_tokens=64, dtype=K.KDA_BF16, input_kind=1),
                 ("d_o", "gate", "o", "x", "state_in", "dstate_out", "dx", "dgate", "dstate_in", "cu_seqlens"), kw)


def _norm(**kw):
    return _fill(K.KdaAddNormArgs(total_tokens=8, channels=256, dtype=K.KDA_BF16, quant=2, eps=1e-6),
                 ("x", "residual", "weight", "residual_out", "y", "scale"), kw)


def _norm_grad(**kw):
    kw = dict({"workspace_bytes": 1 << 20}, **kw)
    return _fill(K.KdaAddNormBackwardArgs(total_tokens=8, channels=256, dtype=K.KDA_BF16, eps=1e-6),
                 ("dy", "s", "dresidual", "weight", "dx", "dweight", "workspace"), kw)


SHARED = [({"num_seqs": 0}, INV), ({"channels": 0}, INV), ({"channels": -8}, INV), ({"channels": 76}, INV),
          ({"dtype": 2}, INV), ({"gate_kind": 2}, INV), ({"gate_kind": -1}, INV), ({"input_kind": 3}, INV),
          ({"flags": 1}, UNS), ({"flags": 256}, UNS), ({"num_seqs": 1 << 22}, INV), ({"gate": None}, INV),
          ({"o": None}, INV), ({"gate": _addr(1) + 8}, INV), ({"gate_stride": 71}, INV), ({"gate_stride": 76}, INV),
          ({"o_stride": -72}, INV), ({"gate_stride": 1 << 50}, INV)]
WIDE = [({"gate_stride": (1 << 22) + 8}, UNS), ({"o_stride": (1 << 22) + 8}, UNS)]
FORWARD = [({"x": None}, INV), ({"x": _addr(0) + 2}, INV), ({"x_stride": 64}, INV), ({"o": _addr(0)}, INV),
           ({"o": _addr(1) + 16}, INV), ({"state_slots": _addr(9)}, INV),
           ({"state_slots": _addr(9), "num_slots": -1}, INV), ({"state_slots": _addr(4), "num_slots": 4}, INV)]
TOKENS = [({"total_tokens": -1}, INV), ({"total_tokens": 1 << 31}, INV), ({"total_tokens": (1 << 31) - 511}, INV),
          ({"total_tokens": 65, "cu_seqlens": None}, INV),
          ({"schedule": 2}, UNS), ({"schedule": 3}, UNS), ({"schedule": 5}, UNS), ({"schedule": -1}, UNS),
          ({"schedule": 4}, INV), ({"schedule": 4, "workspace": _addr(20), "workspace_bytes": 64}, INV),
          ({"schedule": 4, "workspace": _addr(20) + 8, "workspace_bytes": 1 << 20}, INV)]


@pytest.mark.parametrize("kw,status", SHARED + WIDE + FORWARD + TOKENS + [
    ({"state_out": _addr(2) + 64}, INV), ({"state_out": _addr(0)}, INV), ({"state_in": _addr(2) + 4}, INV),
    ({"state_out": _addr(5)}, INV), ({"state_in": _addr(4)}, INV), ({"cu_seqlens": _addr(4)}, INV),
    ({"schedule": 4, "workspace": _addr(0), "workspace_bytes": 1 << 20}, INV),
    ({"schedule": 4, "workspace": _addr(4), "workspace_bytes": 1 << 20}, INV)])
def test_prefill_refusals(lib, kw, status):
    assert lib.kda_gated_scan_prefill(ctypes.byref(_scan(**kw)), None) == status
    assert lib.kda_last_error() != b""


@pytest.mark.parametrize("kw,status", SHARED + FORWARD[:-1] + [
    ({"state": None}, INV), ({"state": _addr(2) + 8}, INV), ({"state": _addr(3)}, INV), ({"state": _addr(0)}, INV)])
def test_decode_refusals(lib, kw, status):
    assert lib.kda_gated_scan_decode(ctypes.byref(_step(**kw)), None) == status
    assert lib.kda_last_error() != b""


@pytest.mark.parametrize("kw,status", SHARED + WIDE + TOKENS + [
    ({"x": None}, INV), ({"input_kind": 0}, INV), ({"d_o": None}, INV), ({"dx": None}, INV), ({"dgate": None}, INV),
    ({"dx": _addr(0)}, INV), ({"dgate": _addr(6)}, INV), ({"dgate": _addr(1)}, INV), ({"dx": _addr(2)}, INV),
    ({"dx": _addr(3)}, INV), ({"dstate_in": _addr(6)}, INV), ({"dstate_in": _addr(4)}, INV),
    ({"dstate_in": _addr(5) + 64}, INV), ({"dstate_out": _addr(5) + 8}, INV), ({"dx_stride": 68}, INV),
    ({"d_o": _addr(0) + 4}, INV), ({"dstate_in": _addr(9)}, INV)])
def test_backward_refusals(lib, kw, status):
    assert lib.kda_gated_scan_backward(ctypes.byref(_grad(**kw)), None) == status
    assert lib.kda_last_error() != b""


def test_host_lengths_are_checked(lib):
    for make, f in ((_scan, lib.kda_gated_scan_prefill), (_grad, lib.kda_gated_scan_backward)):
        for cu in ([1, 30, 64], [0, 70, 64], [0, 30, 63]):
            arr = (ctypes.c_int32 * 3)(*cu)
            assert f(ctypes.byref(make(cu_seqlens_host=ctypes.cast(arr, ctypes.c_void_p))), None) == INV, cu
        arr = (ctypes.c_int32 * 3)(0, 30, 64)
        assert f(ctypes.byref(make(cu_seqlens=None, cu_seqlens_host=ctypes.cast(arr, ctypes.c_void_p))), None) == INV


@pytest.mark.parametrize("kw,status", [
    ({"total_tokens": -1}, INV), ({"total_tokens": 1 << 31}, INV), ({"channels": 0}, UNS), ({"channels": 252}, UNS),
    ({"channels": 16392}, UNS), ({"channels": 264}, UNS), ({"dtype": 3}, INV), ({"quant": 3}, INV), ({"quant": -1}, INV),
    ({"quant": 0}, INV), ({"scale": None}, INV), ({"eps": 0.0}, INV), ({"eps": float("nan")}, INV), ({"x": None}, INV),
    ({"y": None}, INV), ({"x": _addr(0) + 8}, INV), ({"y": _addr(4) + 4}, INV), ({"y_stride": 260}, INV),
    ({"x_stride": 255}, INV), ({"residual_stride": 260}, INV), ({"weight": _addr(2) + 4}, INV),
    ({"scale": _addr(5) + 2}, INV), ({"y": _addr(0)}, INV), ({"y": _addr(3)}, INV), ({"residual_out": _addr(0) + 16}, INV),
    ({"residual_out": _addr(1), "residual_out_stride": 264}, INV), ({"scale": _addr(4)}, INV), ({"scale": _addr(2)}, INV),
    ({"residual_out": _addr(2)}, INV), ({"y": _addr(2)}, INV)])
def test_add_norm_refusals(lib, kw, status):
    assert lib.kda_add_norm(ctypes.byref(_norm(**kw)), None) == status
    assert lib.kda_last_error() != b""


@pytest.mark.parametrize("kw,status", [
    ({"total_tokens": -1}, INV), ({"channels": 4}, UNS), ({"channels": 16392}, UNS), ({"dtype": 2}, INV),
    ({"eps": -1.0}, INV), ({"dy": None}, INV), ({"s": None}, INV), ({"dx": None}, INV), ({"workspace": None}, INV),
    ({"workspace_bytes": 2 * 256 * 4 - 1}, INV), ({"workspace": _addr(6) + 4}, INV), ({"dweight": _addr(5) + 4}, INV),
    ({"weight": _addr(3) + 8}, INV), ({"dx": _addr(0) + 16}, INV), ({"dx": _addr(1), "dx_stride": 264}, INV),
    ({"dx": _addr(3)}, INV), ({"dweight": _addr(4)}, INV), ({"dweight": _addr(3)}, INV), ({"workspace": _addr(0)}, INV),
    ({"dy_stride": 248}, INV), ({"dresidual_stride": 257}, INV)])
def test_add_norm_backward_refusals(lib, kw, status):
    assert lib.kda_add_norm_backward(ctypes.byref(_norm_grad(**kw)), None) == status
    assert lib.kda_last_error() != b""


def test_workspace_sizes(lib):
    def size(backward=False, **kw):
        make, f = (_grad, lib.kda_gated_scan_backward_workspace_size) if backward else (_scan, lib.kda_gated_scan_workspace_size)
        return f(ctypes.byref(make(cu_seqlens=None, num_seqs=1, **kw)))
    for backward in (False, True):
        assert size(backward, total_tokens=0) == 0 and size(backward, total_tokens=-3) == 0
        assert size(backward, total_tokens=64) == 0                     # a tile: nothing to hand on
        assert size(backward, total_tokens=64, schedule=4) > 0          # asked for
        assert size(backward, total_tokens=1 << 16) > 0 and size(backward, total_tokens=1 << 16, schedule=1) == 0
        for T in (1, 239, 240, 241, (1 << 31) - 512):                    # absurd calls stay arithmetic
            for C in (8, 1000, 2147483640):
                size(backward, total_tokens=T, channels=C, schedule=4)
    assert size(total_tokens=(1 << 31) - 512, schedule=4, channels=8) == 0  # too many tiles for a launch
    a = _scan(cu_seqlens=None, num_seqs=1, total_tokens=(1 << 31) - 512, channels=8, schedule=4, workspace=1 << 60,
              workspace_bytes=1 << 60, x=_addr(1 << 10), gate=_addr(1 << 12), o=_addr(1 << 14))
    assert lib.kda_gated_scan_prefill(ctypes.byref(a), None) == INV and b"tiles" in lib.kda_last_error()
    assert lib.kda_gated_scan_workspace_size(None) == 0 and lib.kda_gated_scan_backward_workspace_size(None) == 0
    assert lib.kda_add_norm_backward_workspace_size(None) == 0
    assert lib.kda_add_norm_backward_workspace_size(ctypes.byref(_norm_grad(dweight=None))) == 0
    assert lib.kda_add_norm_backward_workspace_size(ctypes.byref(_norm_grad())) == 2 * 256 * 4


def test_null_arguments_and_nothing_to_do(lib):
    for f in ("kda_gated_scan_prefill", "kda_gated_scan_decode", "kda_gated_scan_backward", "kda_add_norm",
              "kda_add_norm_backward"):
        assert getattr(lib, f)(None, None) == INV
    for sched in (0, 1, 4):
        assert lib.kda_gated_scan_prefill(ctypes.byref(_scan(total_tokens=0, state_out=None, schedule=sched)), None) == 0
        assert lib.kda_gated_scan_backward(ctypes.byref(_grad(total_tokens=0, dstate_in=None, schedule=sched)), None) == 0
    assert lib.kda_add_norm(ctypes.byref(_norm(total_tokens=0, x=None)), None) == 0
    assert lib.kda_add_norm_backward(ctypes.byref(_norm_grad(total_tokens=0, dy=None, dweight=None)), None) == 0


def test_struct_sizes():
    for pack, s, ws in ((K._SCAN_PACK, K.KdaGatedScanArgs, True), (K._STEP_PACK, K.KdaGatedScanDecodeArgs, False),
                        (K._SCAN_GRAD_PACK, K.KdaGatedScanBackwardArgs, True), (K._ADD_NORM_PACK, K.KdaAddNormArgs, False),
                        (K._ADD_NORM_GRAD_PACK, K.KdaAddNormBackwardArgs, True)):
        assert pack.size + (K._WORKSPACE_PACK.size if ws else 0) == ctypes.sizeof(s)
        assert not ws or s.workspace.offset == pack.size
    assert K.KdaGatedScanArgs.x.offset == 56 and K.KdaGatedScanDecodeArgs.x.offset == 48
    assert K.KdaGatedScanBackwardArgs.d_o.offset == 80 and K.KdaAddNormArgs.x.offset == 56
    assert K.KdaAddNormBackwardArgs.dy.offset == 56


# ------------------------------------------------------------------ the Python binding
def test_python_refuses_cpu_tensors():
    x, s = torch.zeros(6, 16), torch.zeros(6, 16)
    for call in (lambda: kda.kda_gated_scan_prefill(x, x), lambda: kda.kda_gated_scan_decode(x, x, s),
                 lambda: kda.kda_gated_scan_backward(x, x, x), lambda: kda.kda_add_norm(x, x),
                 lambda: kda.kda_add_norm_backward(x, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_python_checks_scan_tensors():
    x, g = torch.zeros(6, 16, dtype=BF), torch.zeros(6, 16, dtype=BF)
    st, slots = torch.zeros(1, 16), torch.zeros(1, dtype=torch.int32)
    for bad, err, match in [
            (dict(x=x[0]), ValueError, "x must be"), (dict(g=g[:, :8]), ValueError, "gate must have"),
            (dict(g=g.float()), TypeError, "gate must be"), (dict(x=x.t().contiguous().t()), ValueError, "dense"),
            (dict(x=x[:1].expand(6, 16)), ValueError, "overlap"), (dict(gate_kind="exp"), ValueError, "gate_kind"),
            (dict(input_kind="none"), ValueError, "input_kind"), (dict(schedule="two_pass"), ValueError, "schedule"),
            (dict(state_in=st, num_seqs=0), ValueError, "state_in"),
            (dict(state_in=torch.zeros(2, 16)), ValueError, "state_in"), (dict(state_in=st.double()), TypeError, "state"),
            (dict(state_in=st, state_out=st.bfloat16()), TypeError, "one dtype"), (dict(o=x.float()), TypeError, "o must be"),
            (dict(cu_seqlens=torch.tensor([0, 6])), TypeError, "cu_seqlens"),
            (dict(cu_seqlens=torch.tensor([0, 6], dtype=torch.int32), cu_seqlens_host=[0, 3, 6]), ValueError, "host"),
            (dict(state_slots=slots), ValueError, "pool"), (dict(state_slots=slots, state_in=st, state_out=True), ValueError, "pool"),
            (dict(state_slots=slots.repeat(2), state_in=st), ValueError, "one slot"),
            (dict(state_slots=slots.float(), state_in=st), TypeError, "state_slots"),
            (dict(workspace=torch.zeros(64)), TypeError, "workspace"), (dict(x=x.half(), g=g.half()), TypeError, "unsupported dtype")]:
        kw = dict(x=x, g=g)
        kw.update(bad)
        with pytest.raises(err, match=match):
            kda.kda_gated_scan_prefill(kw.pop("x"), kw.pop("g"), **kw)
    with pytest.raises(ValueError, match="one row"):
        kda.kda_gated_scan_decode(x, g, st)
    with pytest.raises(ValueError, match="state must have"):
        kda.kda_gated_scan_decode(x, g, torch.zeros(6, 8))
    for bad, err, match in [
            (dict(x=x), ValueError, "x goes"), (dict(input_kind="norm"), ValueError, "x goes"),
            (dict(o=x[:5]), ValueError, "o must have"), (dict(dx=x.float()), TypeError, "dx"),
            (dict(dgate=x[:, :8]), ValueError, "dgate"), (dict(dstate_out=st.bfloat16()), TypeError, "dstate_out"),
            (dict(dstate_in=torch.zeros(2, 16)), ValueError, "dstate_in"), (dict(state_in=torch.zeros(2, 16)), ValueError, "state_in")]:
        kw = dict(d=x, g=g, o=x)
        kw.update(bad)
        with pytest.raises(err, match=match):
            kda.kda_gated_scan_backward(kw.pop("d"), kw.pop("g"), kw.pop("o"), **kw)


def test_python_checks_norm_tensors():
    x, w = torch.zeros(6, 136, dtype=BF), torch.ones(136)
    for bad, err, match in [
            (dict(residual=x[:5]), ValueError, "residual"), (dict(weight=w.double()), TypeError, "weight"),
            (dict(weight=w[:8].clone()), ValueError, "weight"), (dict(quant="int8"), ValueError, "quant"),
            (dict(quant="group"), ValueError, "128"), (dict(scale=torch.ones(6)), ValueError, "scale"),
            (dict(quant="token", scale=torch.ones(5)), ValueError, "scale"), (dict(quant="token", y=x), TypeError, "y must be"),
            (dict(y=x[:, :8]), ValueError, "y must have"), (dict(residual_out=x.float()), TypeError, "residual_out")]:
        with pytest.raises(err, match=match):
            kda.kda_add_norm(x, **bad)
    for bad, err, match in [(dict(s=x[:5]), ValueError, "s must have"), (dict(dresidual=x.float()), TypeError, "dresidual"),
                            (dict(dweight=w.bfloat16()), TypeError, "dweight"), (dict(dx=x[:, :8]), ValueError, "dx"),
                            (dict(workspace=w), TypeError, "workspace")]:
        kw = dict(s=x)
        kw.update(bad)
        with pytest.raises(err, match=match):
            kda.kda_add_norm_backward(x, kw.pop("s"), **kw)


def test_import_on_a_torch_without_gpu_support():
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import gated_delta_rule_short_amd as kda
x = torch.zeros(2, 16)
for call in (lambda: kda.kda_gated_scan_prefill(x, x), lambda: kda.kda_gated_scan_decode(x, x, x.clone()),
             lambda: kda.kda_gated_scan_backward(x, x, x), lambda: kda.kda_add_norm(x),
             lambda: kda.kda_add_norm_backward(x, x)):
    try:
        call()
    except ValueError as e:
        assert "GPU" in str(e), e
    else:
        raise AssertionError("accepted")
print("refused")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr[-2000:]


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is needed for the C ABI build")
def test_host_code_under_address_and_undefined_sanitizers(tmp_path):
    src, csrc = os.path.join(ROOT, "tests", "sanitize"), os.path.join(ROOT, "gated_delta_rule_short_amd", "csrc")
    flags = ["-std=c++17", "-g", "-O1", "-fno-omit-frame-pointer", "-Xarch_host", "-fsanitize=address",
             "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all",
             "-I" + os.path.join(ROOT, "include"), "-I" + csrc]
    api, drv, exe = (str(tmp_path / n) for n in ("api.o", "driver.o", "asan"))
    for cmd in ([HIPCC, "--offload-arch=gfx950"] + flags + ["-c", os.path.join(csrc, "kda_scan_api.hip"), "-o", api],
                [HIPCC, "-x", "c++", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include"] + flags
                + ["-c", os.path.join(src, "scan_driver.cpp"), "-o", drv],
                [HIPCC, "--offload-arch=gfx950"] + flags[:10] + [api, drv, "-o", exe], [exe]):
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=600,
                           env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
        assert r.returncode == 0, "%s\n%s\n%s" % (" ".join(cmd), r.stdout[-4000:], r.stderr[-4000:])
    assert "scan sanitizer run ok" in r.stdout


def test_a_workspace_too_small_is_refused_under_every_choice_that_uses_it(lib):
    """The automatic choice takes no other schedule for a smaller workspace; one pass, and
    calls that it is right for, need none."""
    for make, size_of, call in (
            (_scan, lib.kda_gated_scan_workspace_size, lib.kda_gated_scan_prefill),
            (_grad, lib.kda_gated_scan_backward_workspace_size, lib.kda_gated_scan_backward)):
        for sched in (0, 4):
            args = dict(cu_seqlens=None, num_seqs=1, total_tokens=1 << 16, schedule=sched, workspace=_addr(20))
            need = size_of(ctypes.byref(make(**args)))
            assert need > 256
            assert call(ctypes.byref(make(workspace_bytes=need - 1, **args)), None) == INV
            assert b"needed" in lib.kda_last_error()
        assert size_of(ctypes.byref(make(cu_seqlens=None, num_seqs=1, total_tokens=1 << 16, schedule=1))) == 0
