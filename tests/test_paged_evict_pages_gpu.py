"""Evictions over tables of more pages than a CTA's threads (1024), which the
choice checks in rounds, and than the move keeps in shared memory (2048); and the
K and V of the sequences beside one that is skipped."""
import numpy as np
import pytest
import torch

import kv_cached_gqa_rope_gb300 as kv
import oracle
from paged_helpers import Paged, bits16
from test_paged_gpu import check_evict, evict

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def masses(A, H_kv, M, seed):
    return (torch.rand(A, H_kv, M, generator=torch.Generator().manual_seed(seed)) ** 4).cuda()


def check_pools(p, mass, keep, recent, skipped):
    """K and V of all sequences; those of `skipped` as they were."""
    kl = [0 if a in skipped else n for a, n in enumerate(p.kl)]
    k, v, _, _, _ = oracle.paged_evict(mass.cpu().numpy(), kl, p.table.numpy(), keep, recent, bits16(p.k_cache),
                                       bits16(p.v_cache))
    assert np.array_equal(bits16(p.d_k_cache), k) and np.array_equal(bits16(p.d_v_cache), v)


@pytest.mark.parametrize("H_kv,D,dtype", [(1, 64, BF), (2, 128, HF)])
def test_sources_and_places_behind_the_kept_table(H_kv, D, dtype):
    n, keep = 40000, 2048 * 16 + 1500
    p = Paged([0], [n], H_kv, H_kv, D, 16, dtype, seed=81).cuda()
    mass = masses(1, H_kv, p.max_pages * 16, 12)
    got = evict(p, mass, keep, 100)
    assert got[3] == 0
    check_evict(p, mass, keep, 100, got)


@pytest.mark.parametrize("page", [1023, 1024, 2047, 2048, 2400])
def test_a_bad_entry_far_back_in_the_table(page):
    """One bad entry anywhere skips its sequence whole, and it alone."""
    p = Paged([0, 0, 0], [700, 2401 * 16, 300], 1, 1, 64, 16, BF, seed=82).cuda()
    mass = masses(3, 1, p.max_pages * 16, 13)
    p.d_table[1, page] = p.P
    got = evict(p, mass, 200, 30)
    assert got[3] == kv.FLAG_PAGE_RANGE
    check_evict(p, mass, 200, 30, got, seqs=[0, 2])
    check_pools(p, mass, 200, 30, [1])
    assert torch.all(got[1][1] == 7) and int(got[2][1]) == 7 and torch.all(got[0][1] == 7)


def test_neighbours_of_a_skipped_sequence_move():
    for bad in ("entry", "length", "mass"):
        p = Paged([0] * 4, [100, 200, 300, 64], 2, 2, 64, 16, HF, seed=83).cuda()
        mass = masses(4, 2, 320, 14)
        skipped = 1
        if bad == "entry":
            p.d_table[1, 12] = -1
        elif bad == "length":
            p.d_lengths[1] = 10 ** 9
        else:
            mass, skipped = mass[:, :, :250].contiguous(), 2      # fewer cells than sequence 2 has
        got = evict(p, mass, 64, 8)
        assert got[3] == (kv.FLAG_PAGE_RANGE if bad == "entry" else kv.FLAG_POSITION_RANGE)
        wide = torch.zeros(4, 2, 320, device="cuda")
        wide[:, :, :mass.shape[2]] = mass
        check_pools(p, wide, 64, 8, [skipped])
