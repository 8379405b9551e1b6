"""Evictions whose mass rows are as wide as a server's longest context, over
sequences of every length."""
import pytest
import torch

from paged_helpers import Paged
from test_paged_gpu import check_evict, evict

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("keep,recent", [(300, 40), (9000, 0)])
def test_short_rows_in_a_wide_mass(keep, recent):
    """The form of the choice goes by each sequence's length: masses in shared
    memory up to 9216 cells, read from L2 beyond, in one call."""
    kl = [500, 9215, 9216, 9217, 20000, 0, 70, 301]
    p = Paged([0] * len(kl), kl, 2, 2, 64, 64, BF, seed=80).cuda()
    g = torch.Generator().manual_seed(11)
    mass = torch.rand(p.A, 2, 40000, generator=g) ** 8
    mass[torch.rand(mass.shape, generator=g) < 0.3] = 0.0        # ties across the border
    for a, n in enumerate(kl):
        mass[a, :, n:] = float("inf")                            # behind a sequence: nothing that counts
    mass = mass.cuda()
    got = evict(p, mass, keep, recent)
    assert got[3] == 0
    check_evict(p, mass, keep, recent, got)
