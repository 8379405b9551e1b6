"""Attention over 8-bit pages whose value scales lie far apart: what a row does
not see, or what weighs next to nothing in it, costs its other values nothing."""
import numpy as np
import pytest
import torch

import oracle
from e4m3_row_bounds import check_rows, problem
from test_e4m3_gpu import attend

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
GAPS = [(BF, 20), (BF, 34), (BF, 60), (HF, 20), (HF, 24)]
TOKENS = [1, 3, 40]
LATER = [(4, 322, 2, 128), (4, 386, 2, 64), (8, 130, 4, 64), (16, 50, 1, 128),
         (40, 322, 4, 128), (40, 386, 4, 64), (150, 258, 2, 64), (300, 338, 2, 128)]


def run(p):
    p.cuda()
    out, lse, flags = attend(p)
    assert flags == 0
    check_rows(p, out, lse)


@pytest.mark.parametrize("dtype,gap", GAPS)
@pytest.mark.parametrize("ql,kl,H_q,D", LATER)
def test_a_later_token_of_the_chunk(ql, kl, H_q, D, dtype, gap):
    """The last two cells, which all rows but the last tokens' do not see."""
    p = problem([ql, 1], [kl, 77], H_q, 1, D, dtype)
    p.v_scale[int(p.table[0, kl // 16])] += gap
    run(p)


def weigh(p, block, nats):
    """The keys of a block of sequence 0, so that its scores are `nats` for every row."""
    codes = p.k_codes
    codes[codes == 127] = 0
    codes[..., 0] = 0
    p.q[..., 0] = 16.0
    pid = int(p.table[0, block])
    codes[pid] = 0
    e = int(oracle.e4m3_exponent(abs(nats) / (16.0 * p.scale)))
    p.k_scale[pid] = e
    codes[pid, ..., 0] = int(oracle.e4m3_codes(nats / (16.0 * p.scale) / oracle.e4m3_scale(e)))


@pytest.mark.parametrize("dtype,gap", GAPS)
@pytest.mark.parametrize("block", [0, 11, 18])
@pytest.mark.parametrize("ql", TOKENS)
def test_cells_of_next_to_no_weight(ql, block, dtype, gap):
    p = problem([ql, 2], [350, 40], 4, 1, 128, dtype, seed=2)
    weigh(p, block, -112.0)
    p.v_scale[int(p.table[0, block])] += gap
    run(p)


@pytest.mark.parametrize("dtype,gap", GAPS)
@pytest.mark.parametrize("block", [0, 11, 18])
@pytest.mark.parametrize("ql", TOKENS)
def test_small_weights_of_large_values(ql, block, dtype, gap):
    """A block whose values outweigh the others' about as much as the others outweigh it."""
    p = problem([ql], [350], 4, 2, 64, dtype, seed=3)
    weigh(p, block, -0.6931 * gap)
    p.v_scale[int(p.table[0, block])] += gap
    run(p)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("block", [0, 11, 18])
@pytest.mark.parametrize("nats", [5.0, 14.0, 40.0])
@pytest.mark.parametrize("ql", TOKENS)
def test_large_weights_of_small_values(ql, nats, block, dtype):
    p = problem([ql], [350], 4, 2, 128, dtype, seed=4)
    weigh(p, block, nats)
    p.v_scale[int(p.table[0, block])] -= 20 if dtype == BF else 6
    run(p)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("ql", [1, 40])
def test_blocks_of_scale_zero(ql, dtype):
    """The first two tiles, single blocks, and all of a sequence."""
    p = problem([ql, ql, ql], [500, 400, 300], 4, 2, 64, dtype, seed=5)
    p.v_scale[p.table[0, :17].long()] = 0
    p.v_scale[p.table[1, 5:7].long()] = 0
    p.v_scale[p.table[2, :19].long()] = 0
    run(p)


@pytest.mark.parametrize("dtype,gap", [(BF, 34), (HF, 24)])
@pytest.mark.parametrize("ql", TOKENS)
def test_parts_of_many_ctas(ql, dtype, gap):
    """One head's tiles over many CTAs: the parts with the large values and those without."""
    p = problem([ql], [20000], 2, 1, 128, dtype, seed=7)
    weigh(p, 700, -112.0)
    p.v_scale[int(p.table[0, 700])] += gap
    p.v_scale[int(p.table[0, 1249])] += gap                      # the last 16 cells
    run(p)
