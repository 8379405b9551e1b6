"""Decode steps over 8-bit pages of more sequences than a CTA keeps at hand, and
than it has threads."""
import pytest
import torch

from e4m3_helpers import Codes
from test_e4m3_gpu import attend, check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("A", [31, 32, 33, 479, 480, 481, 1100])
@pytest.mark.parametrize("H_q,H_kv,D,dtype", [(8, 2, 64, torch.bfloat16), (3, 1, 128, torch.float16)])
def test_many_sequences(A, H_q, H_kv, D, dtype):
    ql = [0 if i % 7 == 3 else 1 for i in range(A)]
    kl = [1 + i * 37 % 400 for i in range(A)]
    p = Codes(ql, kl, H_q, H_kv, D, 16, dtype, seed=A, behind=A % 3).cuda()
    out, lse, flags = attend(p)
    assert flags == 0
    check_attention(p, out, lse)
    for _ in range(10):
        again, lse2, flags = attend(p)
        assert flags == 0 and torch.equal(out, again) and torch.equal(lse, lse2)
