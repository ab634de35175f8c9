"""The linear-attention entry points at the edges of what the binding and the checks
accept, without a GPU: calls with nothing to do, and a torch build that knows no GPU."""
import ctypes
import os
import subprocess
import sys

import pytest

from gated_delta_rule_short_amd import kda as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(K.LIB_PATH):
        from gated_delta_rule_short_amd import _build
        _build.build()
    return K.load_library()


@pytest.mark.parametrize("schedule", [0, 1, 2])
def test_an_empty_batch_needs_no_workspace(lib, schedule):
    """A batch without tokens runs no passes, whichever schedule is asked for: the size
    is 0 and the call with none is accepted."""
    a = K.KdaLinattnPrefillArgs(num_seqs=2, num_heads=4, num_k_heads=2, head_dim_k=128, head_dim_v=64,
                                dtype=K.KDA_BF16, total_tokens=0, schedule=schedule)
    assert lib.kda_linattn_workspace_size(ctypes.byref(a)) == 0
    assert lib.kda_linattn_prefill(ctypes.byref(a), None) == K.KDA_OK


def test_import_on_a_torch_without_gpu_support():
    """A torch build without GPU support lacks its device and stream functions: the package
    still imports, and host tensors are refused as elsewhere."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import gated_delta_rule_short_amd as kda
q = torch.zeros(2, 1, 64)
for call in (lambda: kda.kda_gated_norm(q), lambda: kda.kda_qk_norm_rope(q, q),
             lambda: kda.kda_linattn_prefill(q, q, q, torch.zeros(2, 1)),
             lambda: kda.kda_linattn_decode(q, q, q, torch.zeros(2, 1), torch.zeros(2, 1, 64, 64))):
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
