"""A key cache whose head width is not the queries' is refused by every call
that reads it (its tensor map is made for the queries' width)."""
import pytest
import torch

import kv_cached_gqa_rope_gb300 as kv
from test_abi_host import attention_args, code_of, prefill_args, step_args, varlen_args

BF = torch.bfloat16


def narrow(t):
    return torch.zeros(*t.shape[:-1], 128 if t.shape[-1] == 64 else 64, dtype=t.dtype)


@pytest.mark.parametrize("fn,args", [
    (kv.cached_gqa_attention_out_, attention_args), (kv.decode_step_out_, step_args),
    (kv.decode_step_single_launch_out_, step_args), (kv.prefill_gqa_cached_rows_out_, prefill_args),
    (kv.prefill_varlen_gqa_cached_rows_out_, varlen_args)])
def test_cache_of_another_head_width_is_refused(fn, args):
    a = args()
    assert code_of(fn, **dict(a, k_cache=narrow(a["k_cache"]))) == "EINVAL"


def test_static_scratch_cache_of_another_head_width_is_refused():
    a = attention_args()
    a.pop("workspace")
    assert code_of(kv.cached_gqa_attention_static_scratch_out_, **dict(a, k_cache=narrow(a["k_cache"]))) == "EINVAL"
