"""As many rows as an int counts."""

import pytest
import torch

from test_gpu_few_bits import check_norm, ok

pytestmark = pytest.mark.gpu


def test_norm_of_two_to_the_31_rows_less_one():
    """T = 2^31 - 1 rows of 8 columns, in place: the first, the last and those on either side of 2^30 and of the last
    whole CTA of rows."""
    from mla_absorbed_decode_absorb_gb300 import ops
    T, D = 2 ** 31 - 1, 8
    x = torch.full((T, D), 3.0, dtype=torch.bfloat16, device="cuda")
    w = torch.linspace(0.5, 1.5, D, device="cuda").to(torch.bfloat16)
    rows = torch.tensor([0, 1, 2 ** 30 - 1, 2 ** 30, T - 9, T - 8, T - 7, T - 2, T - 1], device="cuda")
    some = torch.randn(len(rows), D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    x[rows] = some
    ops.mla_rms_norm(x, w, 1e-6, y=x)
    check_norm(some, None, w, 1e-6, y=x[rows])
    assert not (x[:, 0] == 3.0).any()
    ok()
