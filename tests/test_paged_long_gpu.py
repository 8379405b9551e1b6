"""Sequences whose parts lie on dozens of CTAs, against the oracle: single tokens
over a long cache, whose parts the last CTA merges, and a chunk over one, whose
parts a second kernel merges."""
import pytest
import torch

import oracle
from paged_helpers import Paged, assert_within, attention_bounds
from test_paged_gpu import add_mass, attend, check_mass

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("ql,kl,H_q,H_kv,D,page,dtype", [
    ([1], [40000], 4, 1, 128, 64, BF),                  # one head's 313 key tiles on up to 79 CTAs
    ([2, 1, 1], [30000, 77, 20011], 4, 2, 64, 16, HF),
    ([1, 33], [25000, 24033], 2, 2, 128, 32, BF),
    ([1, 200], [500, 20200], 2, 1, 64, 256, HF)])
def test_parts_of_many_ctas(ql, kl, H_q, H_kv, D, page, dtype):
    p = Paged(ql, kl, H_q, H_kv, D, page, dtype, seed=D + page + len(ql)).cuda()
    ref = oracle.paged_attention(p.q.double().numpy(), *p.pools(), p.starts.numpy(), p.kl, p.table.numpy(), p.scale)
    b_out, b_lse = attention_bounds(ref, dtype, max(kl))
    out, lse, flags = attend(p)
    assert flags == 0
    assert_within(out, ref[0], b_out, "out")
    assert_within(lse, ref[1], b_lse, "lse")
    for _ in range(30):
        again, lse2, flags = attend(p)
        assert flags == 0 and torch.equal(out, again) and torch.equal(lse, lse2)
    before = torch.rand(p.A, H_kv, max(kl) + 5, generator=torch.Generator().manual_seed(2))
    mass = before.cuda()
    lse32 = torch.tensor(ref[1], dtype=torch.float32)
    assert add_mass(p, lse32.cuda(), mass) == 0
    check_mass(p, mass, before.double().numpy(), lse32.double().numpy(), ref[3])
