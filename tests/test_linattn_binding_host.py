"""The linear-attention entry points at the edges of what the binding and the checks
accept, without a GPU: calls with nothing to do."""
import ctypes
import os

import pytest

from gated_delta_rule_short_amd import kda as K


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
