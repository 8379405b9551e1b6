"""Rows of a query tile past a prompt's end hold whatever the workspace held;
what they were must not reach the rows of the items that follow in the same CTA."""
import pytest
import torch

import kv_cached_gqa_rope_gb300 as kv
import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
def test_nan_in_the_workspace_behind_short_prompts(D):
    # ragged prompts in more items than the GPU has SMs, so that CTAs go from one to the next
    wl = W.scaled_prefill(W.PREFILL, A=24, T=300, H_q=16, H_kv=4, D=D, slots=24, max_seq=512)
    lengths = [1 + (37 * a) % 300 for a in range(wl.A)]
    offsets = [(53 * a) % 200 for a in range(wl.A)]
    inp = W.make_varlen_inputs(wl, offsets, lengths)
    outs = []
    for fill in (0, 255):
        kc, vc = inp.build_cache("cuda")
        ws = kv.new_workspace(kv.prefill_gqa_cached_rows_workspace_size(wl.A, wl.T, wl.H_q, wl.H_kv, wl.D))
        ws[kv.STATUS_BYTES:] = fill                              # 0xFFFF is a NaN of either storage type
        out = torch.zeros(wl.A, wl.T, wl.H_q, wl.D, dtype=torch.bfloat16, device="cuda")
        kv.prefill_varlen_gqa_cached_rows_out_(inp.q.cuda(), inp.k.cuda(), inp.v.cuda(), inp.offsets.cuda(),
                                               inp.lengths.cuda(), inp.cache_rows.cuda(), wl.theta, wl.scale, kc, vc,
                                               out, ws)
        assert kv.kvgqa_read_status(ws) == 0
        outs.append(out)
    assert torch.isfinite(outs[1].float()).all()
    assert torch.equal(outs[0], outs[1])
