"""A decode step whose rows are all out of range, then a good one at once on
the same stream and workspace: the good one's results and both flags."""
import pytest
import torch

import workloads as W
from gpu_helpers import DecodeRun, whole_step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("single", [False, True], ids=["two_launch", "single_launch"])
def test_a_good_step_behind_one_of_bad_rows(single):
    wl = W.DecodeWorkload(name="bad", index=13, slots=6, max_seq=256, A=4, H_q=8, H_kv=2, D=128, theta=10000.0,
                          positions="fixed", fixed_positions=(0, 100, 255, 31), fixed_rows=(5, 0, 3, 1))
    inp = W.make_decode_inputs(wl)
    alone = DecodeRun(inp)
    whole_step(alone, single_launch=single)
    torch.cuda.synchronize()
    assert alone.kv.kvgqa_read_status(alone.ws_step) == 0
    run = DecodeRun(inp)
    good = run.positions, run.cache_rows
    for bad_positions in (-1, wl.max_seq):
        for _ in range(10):
            run.positions, run.cache_rows = torch.full_like(good[0], bad_positions), torch.full_like(good[1], wl.slots)
            torch.cuda.synchronize()
            whole_step(run, single_launch=single)
            run.positions, run.cache_rows = good
            whole_step(run, ws=run.ws_step, single_launch=single)
            torch.cuda.synchronize()
            assert run.kv.kvgqa_read_status(run.ws_step) == run.kv.FLAG_POSITION_RANGE | run.kv.FLAG_ROW_RANGE
            assert torch.equal(run.out.view(torch.int16), alone.out.view(torch.int16))
            assert torch.equal(run.k_cache.view(torch.int16), alone.k_cache.view(torch.int16))
            assert torch.equal(run.v_cache.view(torch.int16), alone.v_cache.view(torch.int16))
