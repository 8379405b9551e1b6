"""Paged calls one behind the other on a stream, each reading what the one
before wrote, without a synchronisation between: the results of the same calls
with one."""
import numpy as np
import pytest
import torch

import kv_cached_gqa_rope_gb300 as kv
from paged_helpers import Paged

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


class Chain:
    """An eviction, the mass of the queries added to its mass_out, and an
    attention over its new_lengths.  With every sequence at most `keep` cells
    long nothing moves: the eviction's outputs are all its first kernel's."""

    def __init__(self, ql, kl, keep, M, seed, bad_entry=False):
        self.p = p = Paged(ql, kl, 8, 2, 64, 16, BF, seed=seed).cuda()
        self.keep = keep
        if bad_entry:  # of a sequence that would have to move cells
            p.d_table[1, 0] = p.P
        self.mass = torch.rand(p.A, 2, M, generator=torch.Generator().manual_seed(seed)).cuda()
        self.mass_out = torch.empty(p.A, 2, M, device="cuda")
        self.kept = torch.empty(p.A, 2, keep, dtype=torch.int32, device="cuda")
        self.new = torch.empty(p.A, dtype=torch.int32, device="cuda")
        self.out = torch.empty_like(p.d_q)
        self.lse = torch.full((p.N, 8), 3.0, device="cuda")
        self.lse_out = torch.empty(p.N, 8, device="cuda")
        self.ws = [kv.new_workspace(n) for n in (
            kv.paged_evict_workspace_size(p.A, 2, keep), kv.paged_attention_mass_workspace_size(),
            kv.paged_gqa_attention_workspace_size(8, 2, 64))]

    def stale(self):
        """What an earlier step may have left in the outputs."""
        self.mass_out.fill_(1e6)
        self.kept.fill_(7)
        self.new.copy_(torch.tensor(self.p.ql, dtype=torch.int32))  # lengths that are valid, and wrong
        self.out.fill_(9.0)
        self.lse_out.fill_(9.0)

    def calls(self, stream, between=lambda: None):
        p = self.p
        kv.paged_evict_out_(self.mass, p.d_lengths, p.d_table, self.keep, 4, p.d_k_cache, p.d_v_cache, self.mass_out,
                            self.kept, self.new, self.ws[0], stream=stream)
        between()
        kv.paged_attention_mass_out_(p.d_q, self.lse, p.d_k_cache, p.d_starts, p.d_lengths, p.d_table, p.max_query_len,
                                     p.scale, self.mass_out, self.ws[1], stream=stream)
        between()
        kv.paged_gqa_attention_out_(p.d_q, p.d_k_cache, p.d_v_cache, p.d_starts, self.new, p.d_table, p.max_query_len,
                                    p.scale, self.out, self.lse_out, self.ws[2], stream=stream)

    def results(self):
        torch.cuda.synchronize()
        flags = [kv.kvgqa_read_status(w) for w in self.ws]
        return [t.cpu().clone() for t in (self.mass_out, self.kept, self.new, self.out, self.lse_out)], flags


@pytest.mark.parametrize("ql,kl,keep,M,bad_entry", [
    ([1], [40], 64, 400000, False),                     # one sequence, two heads: a move grid that is gone at once
    ([1, 20, 3], [60, 64, 3], 64, 200000, False),
    ([1, 1], [30, 90], 64, 200000, True)])               # the only sequence above keep is skipped
def test_an_eviction_that_moves_nothing(ql, kl, keep, M, bad_entry):
    c = Chain(ql, kl, keep, M, 7, bad_entry)
    stream = torch.cuda.Stream()
    c.stale()
    torch.cuda.synchronize()
    c.calls(stream, torch.cuda.synchronize)
    want, flags = c.results()
    assert flags[0] == (kv.FLAG_PAGE_RANGE if bad_entry else 0)
    if not bad_entry:
        assert flags == [0, 0, 0] and want[2].tolist() == kl
        assert np.array_equal(want[1][0, 0, :kl[0]].numpy(), np.arange(kl[0]))
    for _ in range(20):
        c.stale()
        torch.cuda.synchronize()
        c.calls(stream)
        got, again = c.results()
        assert again == flags and all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        c.calls(stream)
    for _ in range(20):
        c.stale()
        graph.replay()
        got, again = c.results()
        assert again == flags and all(torch.equal(a, b) for a, b in zip(want, got))
