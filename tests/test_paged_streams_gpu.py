"""The paged calls and the slot cache's at once, each on a stream and a workspace
of its own: the results of the same calls one by one."""
import pytest
import torch

import kv_cached_gqa_rope_gb300 as kv
from paged_helpers import Paged

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def paged_job(p, keep):
    """Store, attention, mass and eviction on copies of one problem's pools."""
    axis = kv.rope_axis_of_pair((p.D // 2,))
    positions = torch.arange(p.N, dtype=torch.int32).view(1, -1).cuda()
    M = p.max_pages * p.page
    b = dict(k=p.d_k_cache.clone(), v=p.d_v_cache.clone(), q_rot=torch.empty_like(p.d_q), out=torch.empty_like(p.d_q),
             lse=torch.empty(p.N, p.H_q, device="cuda"), mass=torch.zeros(p.A, p.H_kv, M, device="cuda"),
             mass_out=torch.empty(p.A, p.H_kv, M, device="cuda"),
             kept=torch.empty(p.A, p.H_kv, keep, dtype=torch.int32, device="cuda"),
             new=torch.empty(p.A, dtype=torch.int32, device="cuda"))
    ws = [kv.new_workspace(n) for n in (
        kv.paged_rope_kv_store_workspace_size(), kv.paged_gqa_attention_workspace_size(p.H_q, p.H_kv, p.D),
        kv.paged_attention_mass_workspace_size(), kv.paged_evict_workspace_size(p.A, p.H_kv, keep))]

    def run(stream):
        with torch.cuda.stream(stream):
            b["k"].copy_(p.d_k_cache)
            b["v"].copy_(p.d_v_cache)
            b["mass"].zero_()
        kv.paged_rope_kv_store_out_(p.d_q, p.d_k, p.d_v, positions, *p.meta, 1e4, axis, b["q_rot"], b["k"], b["v"],
                                    ws[0], stream=stream)
        kv.paged_gqa_attention_out_(b["q_rot"], b["k"], b["v"], *p.meta, p.max_query_len, p.scale, b["out"], b["lse"],
                                    ws[1], stream=stream)
        kv.paged_attention_mass_out_(b["q_rot"], b["lse"], b["k"], *p.meta, p.max_query_len, p.scale, b["mass"], ws[2],
                                     stream=stream)
        kv.paged_evict_out_(b["mass"], p.d_lengths, p.d_table, keep, keep // 8, b["k"], b["v"], b["mass_out"], b["kept"],
                            b["new"], ws[3], stream=stream)

    return run, list(b.values()), ws


def slot_job(dtype, D):
    A, H_q, H_kv, L = 6, 8, 2, 1024
    g = torch.Generator().manual_seed(D)
    kc, vc = (torch.randn(A, H_kv, L, D, generator=g).to(dtype).cuda() for _ in range(2))
    q = torch.randn(A, H_q, D, generator=g).to(dtype).cuda()
    positions = torch.tensor([0, 100, 1023, 500, 333, 7], dtype=torch.int32).cuda()
    rows = torch.arange(A, dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    ws = [kv.new_workspace(kv.cached_gqa_attention_workspace_size(A, H_q, H_kv, D))]
    return (lambda stream: kv.cached_gqa_attention_out_(q, kc, vc, positions, rows, D ** -0.5, out, ws[0], stream=stream),
            [out], ws)


def test_everything_at_once():
    jobs = [paged_job(Paged([1, 1, 1], [700, 90, 2000], 8, 2, 64, 16, HF, seed=1).cuda(), 64),
            paged_job(Paged([40, 1, 300], [900, 33, 700], 16, 4, 128, 32, BF, seed=2).cuda(), 128),
            paged_job(Paged([64, 64], [3000, 1000], 8, 2, 64, 64, BF, seed=3).cuda(), 200),
            slot_job(BF, 128), slot_job(HF, 64)]
    for run, _, _ in jobs:
        run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = [[t.clone() for t in outs] for _, outs, _ in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(30):
        for (run, _, _), s in zip(jobs, streams):
            run(s)
    torch.cuda.synchronize()
    for (_, outs, ws), ref in zip(jobs, want):
        assert [kv.kvgqa_read_status(w) for w in ws] == [0] * len(ws)
        for a, b in zip(outs, ref):
            if a.dtype in (BF, HF):
                a, b = a.view(torch.int16), b.view(torch.int16)
            assert torch.equal(a, b)
