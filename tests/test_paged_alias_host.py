"""Operands that must not share memory, one pair at a time, and empty operands of
the slot cache's calls."""
import pytest
import torch

import kv_cached_gqa_rope_gb300 as kv
import test_abi_host as slot
from test_paged_host import PAST_THE_CHECKS, attention_args, code_of, evict_args, store_args

I32 = torch.int32


@pytest.mark.parametrize("fn,args", [(kv.paged_rope_kv_store_out_, store_args), (kv.paged_evict_out_, evict_args)])
def test_calls_that_write_both_pools_want_two(fn, args):
    a = args()
    assert code_of(fn, **dict(a, v_cache=a["k_cache"])) == "EALIAS"


def test_the_attention_may_read_one_pool_twice():
    a = attention_args()
    assert code_of(kv.paged_gqa_attention_out_, **dict(a, v_cache=a["k_cache"])) in PAST_THE_CHECKS


def test_slot_calls_without_rows_take_any_stride():
    """An operand without elements says nothing with its strides."""
    for fn, args, names in ((kv.decode_step_out_, slot.step_args, ("q", "k", "v", "out")),
                            (kv.cached_gqa_attention_out_, slot.attention_args, ("q_rot", "out"))):
        a = args()
        for n in ("positions", "cache_rows"):
            a[n] = torch.zeros(0, dtype=I32)
        for n in names:
            t = a[n]
            a[n] = torch.zeros(t.shape[0], t.shape[2], t.shape[1], dtype=t.dtype).transpose(1, 2)[:0]
        assert code_of(fn, **a) in PAST_THE_CHECKS
