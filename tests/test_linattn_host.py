"""Refusals of the linear-attention and per-head norm entry points, through the C ABI
and the Python binding.  They return before any HIP call, so they run without a GPU;
the host code also runs under address and undefined-behaviour sanitizers with stub
launchers (tests/sanitize/linattn_driver.cpp)."""
import ctypes
import os
import subprocess

import pytest
import torch

import gated_delta_rule_short_amd as kda
from gated_delta_rule_short_amd import kda as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"
INV, UNS = K.KDA_ERR_INVALID_ARG, K.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        from gated_delta_rule_short_amd import _build
        _build.build()
    return K.load_library()


def _addr(i):
    return 0x100000000 * (i + 1)


def _prefill(**kw):
    a = K.KdaLinattnPrefillArgs(num_seqs=2, num_heads=4, num_k_heads=2, head_dim_k=128, head_dim_v=64,
                                dtype=K.KDA_BF16, total_tokens=64)
    for i, f in enumerate(("q", "k", "v", "log_decay", "state_in", "state_out", "o", "cu_seqlens")):
        setattr(a, f, _addr(i))
    for f, v in kw.items():
        setattr(a, f, v)
    return a


def _decode(**kw):
    a = K.KdaLinattnDecodeArgs(num_seqs=2, num_heads=4, num_k_heads=2, head_dim_k=128, head_dim_v=64,
                               dtype=K.KDA_BF16)
    for i, f in enumerate(("q", "k", "v", "log_decay", "state", "o")):
        setattr(a, f, _addr(i))
    for f, v in kw.items():
        setattr(a, f, v)
    return a


def _qk(**kw):
    a = K.KdaQkNormRopeArgs(total_tokens=8, num_q_heads=4, num_k_heads=2, head_dim=128, rotary_dim=64,
                            dtype=K.KDA_BF16, norm=1, eps=1e-6)
    for i, f in enumerate(("q", "k", "q_out", "k_out", "q_weight", "k_weight", "positions", "inv_freq")):
        setattr(a, f, _addr(i))
    for f, v in kw.items():
        setattr(a, f, v)
    return a


def _gated(**kw):
    a = K.KdaGatedNormArgs(total_tokens=8, num_heads=4, head_dim=128, dtype=K.KDA_BF16, eps=1e-6)
    for i, f in enumerate(("x", "z", "weight", "y")):
        setattr(a, f, _addr(i))
    for f, v in kw.items():
        setattr(a, f, v)
    return a


SHARED = [({"num_seqs": 0}, INV), ({"num_heads": 0}, INV), ({"num_k_heads": 0}, INV), ({"num_k_heads": 3}, INV),
          ({"num_k_heads": -2}, INV), ({"head_dim_k": 32}, UNS), ({"head_dim_v": 256}, UNS), ({"dtype": 2}, INV),
          ({"flags": 1}, UNS), ({"flags": 4096}, UNS), ({"scale": -1.0}, INV), ({"scale": float("nan")}, INV),
          ({"num_seqs": 1 << 20}, INV), ({"q": None}, INV), ({"v": None}, INV), ({"o": None}, INV),
          ({"log_decay": None}, INV), ({"q": _addr(0) + 8}, INV), ({"o": _addr(6) + 2}, INV),
          ({"q_stride": 255}, INV), ({"k_stride": 260}, INV), ({"v_stride": -256}, INV), ({"v_stride": 1 << 50}, INV),
          ({"state_slots": _addr(9)}, INV), ({"state_slots": _addr(9), "num_slots": -1}, INV),
          ({"o": _addr(0)}, INV), ({"o": _addr(2) + 16}, INV), ({"o": _addr(3)}, INV)]


@pytest.mark.parametrize("kw,status", SHARED + [
    ({"total_tokens": -1}, INV), ({"total_tokens": 1 << 31}, INV), ({"total_tokens": 65, "cu_seqlens": None}, INV),
    ({"state_out": _addr(4) + 64}, INV), ({"state_out": _addr(0)}, INV), ({"state_in": _addr(4) + 4}, INV),
    ({"state_out": _addr(7)}, INV), ({"o": _addr(4)}, INV)])
def test_prefill_refusals(lib, kw, status):
    a = _prefill(**kw)
    assert lib.kda_linattn_prefill(ctypes.byref(a), None) == status
    assert lib.kda_last_error() != b""


def test_prefill_checks_the_host_lengths(lib):
    for cu in ([1, 30, 64], [0, 70, 64], [0, 30, 63]):
        arr = (ctypes.c_int32 * 3)(*cu)
        a = _prefill(cu_seqlens_host=ctypes.cast(arr, ctypes.c_void_p))
        assert lib.kda_linattn_prefill(ctypes.byref(a), None) == INV, cu
    arr = (ctypes.c_int32 * 3)(0, 30, 64)
    a = _prefill(cu_seqlens=None, cu_seqlens_host=ctypes.cast(arr, ctypes.c_void_p))
    assert lib.kda_linattn_prefill(ctypes.byref(a), None) == INV


@pytest.mark.parametrize("kw,status", SHARED + [({"state": None}, INV), ({"state": _addr(4) + 8}, INV),
                                                ({"state": _addr(5)}, INV), ({"state": _addr(1)}, INV)])
def test_decode_refusals(lib, kw, status):
    a = _decode(**kw)
    assert lib.kda_linattn_decode(ctypes.byref(a), None) == status
    assert lib.kda_last_error() != b""


@pytest.mark.parametrize("kw,status", [
    ({"total_tokens": -1}, INV), ({"total_tokens": 1 << 31}, INV), ({"num_q_heads": 0}, INV),
    ({"num_q_heads": 1 << 20}, INV), ({"num_k_heads": -1}, INV), ({"num_k_heads": 0}, INV), ({"head_dim": 96}, UNS),
    ({"rotary_dim": 8}, UNS), ({"rotary_dim": 144}, UNS), ({"rotary_dim": -16}, UNS), ({"rotary_dim": 0}, INV),
    ({"positions": None}, INV), ({"inv_freq": None}, INV), ({"dtype": 5}, INV), ({"norm": 3}, INV),
    ({"norm": 2}, INV), ({"flags": 1}, UNS), ({"eps": 0.0}, INV), ({"eps": float("inf")}, INV), ({"q": None}, INV),
    ({"k_out": None}, INV), ({"q": _addr(0) + 2}, INV), ({"q_out_stride": 500}, INV), ({"k_stride": 257}, INV),
    ({"q_weight": _addr(4) + 4}, INV), ({"q_out": _addr(0) + 16}, INV), ({"q_out": _addr(0), "q_out_stride": 1024}, INV),
    ({"q_out": _addr(1)}, INV), ({"k_out": _addr(2)}, INV), ({"k_out": _addr(6)}, INV)])
def test_qk_norm_rope_refusals(lib, kw, status):
    a = _qk(**kw)
    assert lib.kda_qk_norm_rope(ctypes.byref(a), None) == status
    assert lib.kda_last_error() != b""


@pytest.mark.parametrize("kw,status", [
    ({"total_tokens": -1}, INV), ({"num_heads": 0}, INV), ({"num_heads": 1 << 20}, INV), ({"head_dim": 256}, UNS),
    ({"dtype": 3}, INV), ({"flags": 2}, UNS), ({"eps": -1.0}, INV), ({"eps": float("nan")}, INV), ({"x": None}, INV),
    ({"y": None}, INV), ({"z": None, "flags": 1}, INV), ({"weight": None, "flags": 1024}, INV),
    ({"x_stride": 511}, INV), ({"z_stride": 516}, INV), ({"y": _addr(3) + 4}, INV), ({"weight": _addr(2) + 8}, INV),
    ({"y": _addr(0) + 32}, INV), ({"y": _addr(1), "y_stride": 520}, INV), ({"y": _addr(2)}, INV)])
def test_gated_norm_refusals(lib, kw, status):
    a = _gated(**kw)
    assert lib.kda_gated_norm(ctypes.byref(a), None) == status
    assert lib.kda_last_error() != b""


def test_workspace_size(lib):
    def size(**kw):
        return lib.kda_linattn_workspace_size(ctypes.byref(_prefill(cu_seqlens=None, num_seqs=1, **kw)))
    assert lib.kda_linattn_workspace_size(None) == 0
    assert size(total_tokens=0) == 0 and size(total_tokens=-5) == 0 and size(total_tokens=1 << 31) == 0
    assert size(total_tokens=128) == 0                      # one pass is the faster one
    assert size(total_tokens=128, schedule=2) > 0           # asked for
    assert size(total_tokens=1 << 20) > 0 and size(total_tokens=1 << 20, schedule=1) == 0
    assert size(total_tokens=1 << 20, schedule=2, num_heads=1 << 21, num_k_heads=1) == 0  # too many pairs
    for T in (1, 63, 64, 65, (1 << 31) - 64):               # sizes far beyond any memory stay arithmetic
        for H in (1, 7, 1 << 19):
            for dtype in (0, 1):
                size(total_tokens=T, schedule=2, num_heads=H, num_k_heads=1, dtype=dtype)


def test_grids_beyond_a_launch_are_refused(lib):
    # blocks of eight key heads: one key head takes the room of eight
    assert lib.kda_linattn_prefill(ctypes.byref(_prefill(num_seqs=1, num_heads=1 << 19, num_k_heads=1)), None) == INV
    ws = dict(workspace=_addr(12), workspace_bytes=1 << 50, schedule=2)
    for N, H in ((1, 1 << 18), (1 << 16, 4)):               # the scan's threads
        a = _prefill(num_seqs=N, num_heads=H, num_k_heads=H, cu_seqlens=None, total_tokens=N * 512, head_dim_k=64,
                     state_in=None, state_out=None, q=_addr(1 << 10), k=_addr(1 << 12), v=_addr(1 << 14),
                     o=_addr(1 << 16), log_decay=_addr(1 << 18), **ws)
        assert lib.kda_linattn_prefill(ctypes.byref(a), None) == INV
        assert b"pairs" in lib.kda_last_error()
        assert lib.kda_linattn_workspace_size(ctypes.byref(a)) == 0


def test_null_arguments(lib):
    for f in ("kda_linattn_prefill", "kda_linattn_decode", "kda_qk_norm_rope", "kda_gated_norm"):
        assert getattr(lib, f)(None, None) == INV


def test_nothing_to_do_is_accepted(lib):
    assert lib.kda_linattn_prefill(ctypes.byref(_prefill(total_tokens=0, state_out=None)), None) == 0
    assert lib.kda_qk_norm_rope(ctypes.byref(_qk(total_tokens=0, q=None)), None) == 0
    assert lib.kda_gated_norm(ctypes.byref(_gated(total_tokens=0, x=None)), None) == 0


def test_struct_sizes(lib):
    assert K.KdaLinattnPrefillArgs.q.offset == 64 and K.KdaLinattnDecodeArgs.q.offset == 56
    assert K.KdaQkNormRopeArgs.q.offset == 72 and K.KdaGatedNormArgs.x.offset == 56


# ------------------------------------------------------------------ the Python binding
def _tensors(T=6, H=4, Hk=2, dk=128, dv=64, dtype=torch.bfloat16):
    return (torch.zeros(T, Hk, dk, dtype=dtype), torch.zeros(T, Hk, dk, dtype=dtype),
            torch.zeros(T, H, dv, dtype=dtype), torch.zeros(T, H))


def test_python_refuses_cpu_tensors():
    q, k, v, g = _tensors()
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_linattn_prefill(q, k, v, g)
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_linattn_decode(q, k, v, g, torch.zeros(6, 4, 128, 64))
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_qk_norm_rope(q, k)
    with pytest.raises(ValueError, match="GPU"):
        kda.kda_gated_norm(v)


def test_python_checks_linattn_tensors():
    q, k, v, g = _tensors()
    st = torch.zeros(1, 4, 128, 64)
    for bad, err, match in [
            (dict(q=q[0]), ValueError, "q must be"), (dict(k=k[:, :1]), ValueError, "k must have"),
            (dict(v=v.float()), TypeError, "v must be"), (dict(q=q.transpose(1, 2)), ValueError, "dense"),
            (dict(v=v[:1].expand(6, 4, 64)), ValueError, "overlap"),
            (dict(v=torch.zeros(6, 4, 128, dtype=v.dtype)[..., :64]), ValueError, "dense"),
            (dict(g=g.double()), TypeError, "log_decay"), (dict(g=g[:, :3]), ValueError, "contiguous"),
            (dict(g=g[0, :3].clone()), ValueError, "log_decay"), (dict(g=g.t().contiguous().t()), ValueError, "contiguous"),
            (dict(state_in=torch.zeros(2, 4, 128, 64)), ValueError, "one row"),
            (dict(state_in=torch.zeros(1, 4, 64, 128)), ValueError, "state_in must have"),
            (dict(state_in=st, state_out=st.bfloat16()), TypeError, "one dtype"),
            (dict(state_in=st.double()), TypeError, "state"),
            (dict(o=torch.zeros(6, 4, 64)), TypeError, "o must be"),
            (dict(cu_seqlens=torch.tensor([0, 6])), TypeError, "cu_seqlens"),
            (dict(cu_seqlens=torch.tensor([0, 6], dtype=torch.int32), cu_seqlens_host=[0, 3, 6]), ValueError, "host"),
            (dict(state_slots=torch.zeros(1, dtype=torch.int32)), ValueError, "pool"),
            (dict(state_slots=torch.zeros(1, dtype=torch.int32), state_in=st, state_out=True), ValueError, "pool"),
            (dict(state_slots=torch.zeros(2, dtype=torch.int32), state_in=st), ValueError, "one slot"),
            (dict(state_slots=torch.zeros(1), state_in=st), TypeError, "state_slots")]:
        kw = dict(q=q, k=k, v=v, g=g)
        kw.update(bad)
        with pytest.raises(err, match=match):
            kda.kda_linattn_prefill(kw.pop("q"), kw.pop("k"), kw.pop("v"), kw.pop("g"), **kw)
    with pytest.raises(ValueError, match="one row"):
        kda.kda_linattn_decode(q, k, v, g, st)
    with pytest.raises(TypeError, match="unsupported dtype"):
        kda.kda_linattn_prefill(q.half(), k.half(), v.half(), g)


def test_python_checks_norm_tensors():
    q, k, v, _ = _tensors()
    pos, fr = torch.zeros(6, dtype=torch.int32), torch.zeros(32)
    for bad, err, match in [
            (dict(k=k[:5]), ValueError, "k must have"), (dict(norm="rmsnorm"), ValueError, "norm"),
            (dict(positions=pos), ValueError, "together"), (dict(positions=pos.long(), inv_freq=fr), TypeError, "positions"),
            (dict(positions=pos[:5], inv_freq=fr), ValueError, "positions"),
            (dict(positions=pos, inv_freq=fr[:0]), ValueError, "inv_freq"),
            (dict(q_weight=torch.ones(64)), ValueError, "q_weight"), (dict(q_out=q.float()), TypeError, "q_out"),
            (dict(k=None, k_weight=torch.ones(128)), ValueError, "need k")]:
        kw = dict(k=k)
        kw.update(bad)
        with pytest.raises(err, match=match):
            kda.kda_qk_norm_rope(q, kw.pop("k"), **kw)
    for bad, err, match in [(dict(gate=v[:, :2]), ValueError, "gate"), (dict(act="relu"), ValueError, "act"),
                            (dict(weight=torch.ones(3, 64)), ValueError, "weight"),
                            (dict(weight=torch.ones(64).double()), TypeError, "weight"),
                            (dict(y=v[:, :, :32]), ValueError, "y must have")]:
        with pytest.raises(err, match=match):
            kda.kda_gated_norm(v, **bad)


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc is needed for the C ABI build")
def test_host_code_under_address_and_undefined_sanitizers(tmp_path):
    src, csrc = os.path.join(ROOT, "tests", "sanitize"), os.path.join(ROOT, "gated_delta_rule_short_amd", "csrc")
    flags = ["-std=c++17", "-g", "-O1", "-fno-omit-frame-pointer", "-Xarch_host", "-fsanitize=address",
             "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all",
             "-I" + os.path.join(ROOT, "include"), "-I" + csrc]
    api, drv, exe = (str(tmp_path / n) for n in ("api.o", "driver.o", "asan"))
    for cmd in ([HIPCC, "--offload-arch=gfx950"] + flags + ["-c", os.path.join(csrc, "kda_linattn_api.hip"), "-o", api],
                [HIPCC, "-x", "c++", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include"] + flags
                + ["-c", os.path.join(src, "linattn_driver.cpp"), "-o", drv],
                [HIPCC, "--offload-arch=gfx950"] + flags[:10] + [api, drv, "-o", exe], [exe]):
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=600,
                           env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
        assert r.returncode == 0, "%s\n%s\n%s" % (" ".join(cmd), r.stdout[-4000:], r.stderr[-4000:])
    assert "linattn sanitizer run ok" in r.stdout
