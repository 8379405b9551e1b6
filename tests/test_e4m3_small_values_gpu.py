"""Attention over 8-bit pages at the lower end of the scales' range: values that
BF16 holds come out, down to the least exponent."""
import pytest
import torch

from e4m3_row_bounds import check_rows, problem
from test_e4m3_gpu import attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ql,kl,H_q,H_kv", [(1, 200, 4, 2), (3, 500, 8, 2), (40, 200, 4, 2), (300, 700, 2, 1), (1, 20000, 1, 1),
                                            (70, 9000, 1, 1)])
@pytest.mark.parametrize("exponent", [1, 4, 9, 14])
def test_scales_near_the_least(ql, kl, H_q, H_kv, exponent):
    p = problem([ql], [kl], H_q, H_kv, 128 if kl < 1000 else 64, torch.bfloat16, seed=exponent)
    p.v_scale[p.table[0, :-(-kl // 16)].long()] = exponent
    p.cuda()
    out, lse, flags = attend(p)
    assert flags == 0
    check_rows(p, out, lse)
