"""The per-head norms over more rows than the workgroups of one launch hold side by
side (2^22 of them): a workgroup's second row, sampled on both sides of the wrap."""
import pytest
import torch

import gated_delta_rule_short_amd as kda
from tests._linattn_common import DEV, check, gated_ref, rope_ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
WRAP = 1 << 22


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    kda.load_library()


def test_qk_norm_rope_second_rows():
    T = WRAP + 5
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.empty(T, 1, 64, dtype=BF, device=DEV).normal_(generator=g)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    fr = (1e6 ** (-2.0 * torch.arange(32, dtype=torch.float64) / 64)).float().to(DEV)
    y, _ = kda.kda_qk_norm_rope(q, positions=pos, inv_freq=fr)
    at = torch.tensor([0, 1, 4, 5, WRAP - 1, WRAP, WRAP + 1, WRAP + 4], device=DEV)
    ref, bound = rope_ref(q[at], None, "rms", 1e-6, pos[at], fr, False)
    check(y[at], ref, bound, "q")


def test_gated_norm_second_rows():
    H, D = 16, 64
    T = WRAP * 32 // H + 3  # 32 rows of 64 to a workgroup
    x = torch.empty(T, H, D, dtype=BF, device=DEV)
    x.fill_(0.5)
    at = torch.tensor([0, 1, 2, 3, T - 4, T - 3, T - 2, T - 1], device=DEV)
    some = torch.randn(8, H, D, generator=torch.Generator().manual_seed(2)).to(BF)
    x[at] = some.to(DEV)
    w = torch.rand(H, D, generator=torch.Generator().manual_seed(3)) + 0.5
    assert kda.kda_gated_norm(x, None, w.to(DEV), eps=1e-5, y=x) is x
    ref, bound = gated_ref(some, None, w, "sigmoid", 1e-5)
    check(x[at], ref, bound, "y")
    ref, bound = gated_ref(torch.full((1, H, D), 0.5, dtype=BF), None, w, "sigmoid", 1e-5)
    check(x[4:5], ref, bound, "the rows between")
