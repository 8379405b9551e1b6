"""query_starts that fall and rise again: every other sequence is flagged, the
rest claim the same rows.  The host's bound of a call's work counts each row
once, so that such sequences together can pass it, and 32 bits with it."""
import pytest
import torch

import kv_cached_gqa_rope_gb300 as kv
from paged_helpers import JUNK, Paged
from test_paged_gpu import add_mass, attend, check_attention

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
N, CELLS, HEADS, PAGE = 16384, 65536, 8, 256


def head_units():
    """The least of a head's units in the kernels' schedules, for a sequence of N
    tokens and CELLS cells: two per key tile that a block of 256 rows sees in the
    attention, one per 256 cells and 128 columns in the mass."""
    attention = sum(2 * ((CELLS - N + 256 * (b + 1)) // 128) for b in range(N // 256))
    return attention, (CELLS // 256) * (N // 128)


# Sequences (the odd ones are the flagged) whose units together pass 2^30; 2^31,
# where a signed sum turns negative; and 2^32, where it comes round to a few.
@pytest.mark.parametrize("A", [5001, 10001, 18701])
def test_work_past_the_schedule_s_units_is_refused(A):
    units = [(A + 1) // 2 * HEADS * u for u in head_units()]
    assert units[0] > {5001: 2 ** 30, 10001: 2 ** 31, 18701: 2 ** 32}[A]
    host = (N // 256 + A) * (CELLS // 128 + N // 128 + 8) * HEADS * 2
    assert host < 2 ** 30                                        # what the call itself can see of it
    starts = torch.zeros(A + 1, dtype=torch.int32)
    starts[1::2] = N
    meta = (starts.cuda(), torch.full((A,), CELLS, dtype=torch.int32, device="cuda"),
            torch.zeros(A, CELLS // PAGE, dtype=torch.int32, device="cuda"))
    q = torch.zeros(N, HEADS, 64, dtype=BF, device="cuda")
    pool = torch.zeros(1, HEADS, PAGE, 64, dtype=BF, device="cuda")
    out = torch.full_like(q, 7.0)
    lse = torch.full((N, HEADS), 7.0, device="cuda")
    ws = kv.new_workspace(kv.paged_gqa_attention_workspace_size(HEADS, HEADS, 64))
    kv.paged_gqa_attention_out_(q, pool, pool.clone(), *meta, N, 0.125, out, lse, ws)
    assert kv.kvgqa_read_status(ws) == kv.FLAG_POSITION_RANGE
    assert torch.all(out == 7.0) and torch.all(lse == 7.0)


def test_mass_past_the_schedule_s_units_is_refused():
    A = 16401                                                    # one mass row of 65536 cells and 4 heads for each: 17 GB
    heads, q_heads = 4, 64
    starts = torch.zeros(A + 1, dtype=torch.int32)
    starts[1::2] = N
    assert (A + 1) // 2 * heads * (CELLS // 256) * (N * 16 // 128) > 2 ** 32
    assert (N * 16 // 128 + A) * (CELLS // 128 + N // 128 + 8) * heads * 2 < 2 ** 30
    meta = (starts.cuda(), torch.full((A,), CELLS, dtype=torch.int32, device="cuda"),
            torch.zeros(A, CELLS // PAGE, dtype=torch.int32, device="cuda"))
    q = torch.zeros(N, q_heads, 64, dtype=BF, device="cuda")
    lse = torch.zeros(N, q_heads, device="cuda")
    pool = torch.zeros(1, heads, PAGE, 64, dtype=BF, device="cuda")
    mass = torch.full((A, heads, CELLS), 7.0, device="cuda")
    ws = kv.new_workspace(kv.paged_attention_mass_workspace_size())
    kv.paged_attention_mass_out_(q, lse, pool, *meta, N, 0.125, mass, ws)
    assert kv.kvgqa_read_status(ws) == kv.FLAG_POSITION_RANGE
    assert mass.min().item() == 7.0 and mass.max().item() == 7.0


def test_overlapping_sequences_are_flagged_and_alone():
    """Sequences 0 and 2 claim rows 0 to 39 and hold the same cells, so that what
    either writes is the same; sequence 1 between them is the flagged one, and
    sequence 3 lies behind."""
    p = Paged([40, 30], [300, 130], 8, 2, 64, 16, BF, seed=70).cuda()
    want, want_lse, flags = attend(p)
    assert flags == 0
    check_attention(p, want, want_lse)
    table = torch.full((4, p.max_pages), JUNK, dtype=torch.int32)
    table[[0, 2]], table[3] = p.table[0], p.table[1]
    p.d_starts = torch.tensor([0, 40, 0, 40, 70], dtype=torch.int32).cuda()
    p.d_lengths = torch.tensor([300, 50, 300, 130], dtype=torch.int32).cuda()
    p.d_table = table.cuda()
    out, lse, flags = attend(p)
    assert flags == kv.FLAG_POSITION_RANGE
    assert torch.all(torch.isfinite(out.float())) and torch.all(torch.isfinite(lse))
    check_attention(p, out, lse)                                 # p's own two sequences, by the oracle
    mass = torch.zeros(4, 2, 304, device="cuda")
    assert add_mass(p, lse, mass) == kv.FLAG_POSITION_RANGE
    assert torch.equal(mass[0], mass[2]) and torch.all(mass[1] == 0)
    total = mass.double().sum(2).cpu()
    assert torch.allclose(total[[0, 3]], torch.tensor([[160.0], [120.0]], dtype=torch.float64), rtol=2e-5)
