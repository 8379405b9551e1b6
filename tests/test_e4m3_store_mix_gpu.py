"""The store into 8-bit pages of steps in which single tokens stand beside prompts,
on both sides of the mean length at which its CTAs take 16 tokens."""
import pytest
import torch

import kv_cached_gqa_rope_gb300 as kv
from e4m3_helpers import Codes
from test_e4m3_gpu import check_store, store

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ql", [[1] * 63 + [700], [1] * 3 + [1021], [1] * 5 + [1600], [1] * 7 + [1600] + [1] * 8, [255] * 3, [256] * 3, [257] * 3,
                                [0, 511, 1, 0]])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_single_tokens_beside_prompts(ql, dtype):
    kl = [n + 7 * i % 53 for i, n in enumerate(ql)]
    p = Codes(ql, kl, 4, 2, 64, 32, dtype, seed=len(ql), behind=3).cuda()
    axis = kv.rope_axis_of_pair((32,))
    positions = torch.arange(p.N, dtype=torch.int32).view(1, -1).cuda()
    q_out, flags = store(p, positions, axis)
    assert flags == 0
    check_store(p, q_out, positions, axis, 10000.0)
