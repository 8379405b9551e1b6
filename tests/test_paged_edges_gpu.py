"""The paged cache's calls at their edges: pools past 32-bit offsets, captured
and replayed small calls, neighbours full of NaN, shared prefix pages, batches
that go from single tokens to chunks and back, no tokens at all."""
import numpy as np
import pytest
import torch

import kv_cached_gqa_rope_gb300 as kv
import oracle
from paged_helpers import JUNK, Paged, assert_within, attention_bounds, bits16
from test_paged_gpu import add_mass, attend, check_attention, check_evict, check_mass, check_store, evict, store

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


def reference(p):
    return oracle.paged_attention(p.q.double().numpy(), *p.pools(), p.starts.numpy(), p.kl, p.table.numpy(), p.scale)


def test_pool_past_32_bit_offsets():
    """The pages of a small problem moved to the end of pools of more than 2^31
    elements each, through every call."""
    p = Paged([1, 70, 3], [300, 130, 3], 8, 4, 128, 128, BF, seed=100).cuda()
    far = 2 ** 31 // (4 * 128 * 128) + 7
    shift = far - p.P
    big = [torch.empty(far, 4, 128, 128, dtype=BF, device="cuda") for _ in range(2)]
    for b, small in zip(big, (p.d_k_cache, p.d_v_cache)):
        assert b.numel() > 2 ** 31
        b[shift:] = small
    table = torch.where(p.table == JUNK, JUNK, p.table + shift).to(torch.int32)
    p.d_k_cache, p.d_v_cache, p.d_table = big[0], big[1], table.cuda()
    out, lse, flags = attend(p)
    assert flags == 0
    check_attention(p, out, lse)
    ref = reference(p)
    before = torch.zeros(3, 4, 512)
    mass = before.cuda()
    assert add_mass(p, torch.tensor(ref[1], dtype=torch.float32).cuda(), mass) == 0
    check_mass(p, mass, before.double().numpy(), ref[1], ref[3])
    axis = kv.rope_axis_of_pair((64,))
    positions = torch.arange(p.N, dtype=torch.int32).view(1, -1).cuda()
    _, flags = store(p, positions, axis)
    assert flags == 0
    p.d_k_cache, p.d_v_cache, p.d_table = big[0][shift:].clone(), big[1][shift:].clone(), p.table.cuda()
    q_out, _ = store(p, positions, axis)                         # the same again near the origin
    assert torch.equal(p.d_k_cache.view(torch.int16), big[0][shift:].view(torch.int16))
    check_store(p, q_out, positions, axis, 10000.0)
    near = evict(p, mass, 100, 10)
    moved = [p.d_k_cache.clone(), p.d_v_cache.clone()]
    p.d_k_cache, p.d_v_cache, p.d_table = big[0], big[1], table.cuda()
    got = evict(p, mass, 100, 10)
    assert got[3] == 0 and all(torch.equal(a, b) for a, b in zip(near[:3], got[:3]))
    for b, m in zip(big, moved):
        assert torch.equal(b[shift:].view(torch.int16), m.view(torch.int16))


def test_small_calls_in_one_graph():
    """A decode step captured twice over in one graph, on one workspace: the
    split sequences' part counts are back at zero in between."""
    p = Paged([1, 1, 2, 0, 1], [2000, 5, 700, 20, 1300], 8, 2, 128, 16, HF, seed=101).cuda()
    want, want_lse, flags = attend(p)
    assert flags == 0
    check_attention(p, want, want_lse)
    ws = kv.new_workspace(kv.paged_gqa_attention_workspace_size(8, 2, 128))
    outs = [torch.zeros_like(want) for _ in range(2)]
    lses = [torch.zeros_like(want_lse) for _ in range(2)]
    stream = torch.cuda.Stream()
    calls = [kv.prepare_paged_gqa_attention_out_(p.d_q, p.d_k_cache, p.d_v_cache, *p.meta, 2, p.scale, o, l, ws,
                                                 stream=stream) for o, l in zip(outs, lses)]
    calls[0]()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for c in calls:
            c()
    for _ in range(50):
        graph.replay()
    torch.cuda.synchronize()
    for o, l in zip(outs, lses):
        assert torch.equal(o, want) and torch.equal(l, want_lse)
    assert kv.kvgqa_read_status(ws) == 0
    counts = ws[kv.STATUS_BYTES:kv.STATUS_BYTES + 32 * 100].view(torch.int32).view(-1, 8)[:, 4]
    assert int(counts.abs().sum()) == 0


def test_whole_step_in_one_graph():
    """Store, attention, mass and eviction captured together and replayed: each
    replay redoes the store into the same cells and evicts what is there."""
    p = Paged([1, 1, 33], [200, 90, 140], 4, 2, 64, 16, BF, seed=102).cuda()
    axis = kv.rope_axis_of_pair((8, 12, 12))
    positions = torch.arange(3 * p.N, dtype=torch.int32).view(3, -1).cuda()
    M = p.max_pages * 16
    keep = 64

    def buffers():
        q_rot = torch.empty_like(p.d_q)
        return dict(q_rot=q_rot, out=torch.empty_like(q_rot), lse=torch.empty(p.N, 4, device="cuda"),
                    mass=torch.zeros(p.A, 2, M, device="cuda"), mass_out=torch.zeros(p.A, 2, M, device="cuda"),
                    kept=torch.zeros(p.A, 2, keep, dtype=torch.int32, device="cuda"),
                    new=torch.zeros(p.A, dtype=torch.int32, device="cuda"), k=p.d_k_cache.clone(), v=p.d_v_cache.clone(),
                    w=[kv.new_workspace(n) for n in (
                        kv.paged_rope_kv_store_workspace_size(), kv.paged_gqa_attention_workspace_size(4, 2, 64),
                        kv.paged_attention_mass_workspace_size(), kv.paged_evict_workspace_size(p.A, 2, keep))])

    def step(b, stream=None):
        kv.paged_rope_kv_store_out_(p.d_q, p.d_k, p.d_v, positions, *p.meta, 1e4, axis, b["q_rot"], b["k"], b["v"],
                                    b["w"][0], stream=stream)
        kv.paged_gqa_attention_out_(b["q_rot"], b["k"], b["v"], *p.meta, 33, p.scale, b["out"], b["lse"], b["w"][1],
                                    stream=stream)
        kv.paged_attention_mass_out_(b["q_rot"], b["lse"], b["k"], *p.meta, 33, p.scale, b["mass"], b["w"][2],
                                     stream=stream)
        kv.paged_evict_out_(b["mass"], p.d_lengths, p.d_table, keep, 16, b["k"], b["v"], b["mass_out"], b["kept"],
                            b["new"], b["w"][3], stream=stream)

    a, b = buffers(), buffers()
    for _ in range(3):
        step(a)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step(b, stream)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for name in ("q_rot", "out", "lse", "mass", "mass_out", "kept", "new"):
        assert torch.equal(a[name], b[name]), name
    assert torch.equal(a["k"].view(torch.int16), b["k"].view(torch.int16))
    assert [kv.kvgqa_read_status(w) for w in a["w"] + b["w"]] == [0] * 8


@pytest.mark.parametrize("ql", [[1, 1, 1, 1], [40, 1, 70, 5], [130, 300, 1, 200]])
def test_a_sequence_of_nan_stays_alone(ql):
    """One sequence's queries, cells and the rows behind the last are all NaN:
    nobody else sees any of it, in the attention or in the mass."""
    kl = [q + n for q, n in zip(ql, (333, 90, 700, 1))]
    p = Paged(ql, kl, 8, 2, 128, 16, BF, seed=103, behind=5)
    nan = float("nan")
    sick = 1
    for i in range(-(-kl[sick] // 16)):
        p.k_cache[int(p.table[sick, i])] = nan
        p.v_cache[int(p.table[sick, i])] = nan
    s, e = int(p.starts[sick]), int(p.starts[sick + 1])
    p.cuda()
    ref = reference(p)                                           # (the sick pages count as zeros there)
    p.d_q[s:e] = nan
    p.d_q[p.live:] = nan
    rows = [n for n in range(p.live) if not s <= n < e]
    out, lse, flags = attend(p)
    assert flags == 0
    check_attention(p, out, lse, rows=rows)
    before = torch.rand(p.A, 2, max(kl) + 1)
    mass = before.cuda()
    assert add_mass(p, torch.tensor(np.nan_to_num(ref[1]), dtype=torch.float32).cuda(), mass) == 0
    check_mass(p, mass, before.double().numpy(), np.nan_to_num(ref[1]), ref[3], seqs=[a for a in range(p.A) if a != sick])


def test_shared_prefix_pages():
    """Sequences that share the pages of a common prefix read them together."""
    p = Paged([5, 1, 60], [133, 129, 200], 8, 2, 64, 32, HF, seed=104)
    for a in (1, 2):
        p.table[a, :4] = p.table[0, :4]                          # 128 cells
    p.cuda()
    out, lse, flags = attend(p)
    assert flags == 0
    check_attention(p, out, lse)


def test_from_single_tokens_to_chunks_and_back():
    """Blocks with one and with two query tiles in every order, over long and
    short prefixes, and the same result from every run."""
    g = np.random.default_rng(5)
    ql = [int(x) for x in g.choice([1, 2, 31, 32, 33, 64, 65, 90, 128, 200], 60)]
    kl = [q + int(x) for q, x in zip(ql, g.choice([0, 1, 127, 128, 500, 1500], 60))]
    p = Paged(ql, kl, 8, 2, 128, 16, BF, seed=105).cuda()
    out, lse, flags = attend(p)
    assert flags == 0
    check_attention(p, out, lse)
    for _ in range(20):
        again, lse2, flags = attend(p)
        assert flags == 0 and torch.equal(out, again) and torch.equal(lse, lse2)


def test_rows_of_no_sequence_and_no_rows():
    p = Paged([0, 0], [5, 0], 4, 2, 64, 16, BF, seed=106, behind=3).cuda()
    out, lse, flags = attend(p, max_query_len=7)
    assert flags == 0 and torch.all(out == 7.0) and torch.all(lse == 7.0)
    mass = torch.ones(2, 2, 32, device="cuda")
    assert add_mass(p, lse, mass, max_query_len=7) == 0 and torch.all(mass == 1)
    q_out, flags = store(p, torch.zeros(1, 3, dtype=torch.int32).cuda(), [0] * 32)
    assert flags == 0 and torch.all(q_out == 7.0)
    assert np.array_equal(bits16(p.d_k_cache), bits16(p.k_cache))
    for behind, A in ((0, 2), (3, 0)):                           # no rows at all; no sequences
        p = Paged([0] * A, [5] * A, 4, 2, 64, 16, BF, seed=107, behind=behind).cuda()
        out, _, flags = attend(p)
        assert flags == 0 and torch.all(out == 7.0)
        _, flags = store(p, torch.zeros(3, p.N, dtype=torch.int32).cuda(), [0] * 32)
        assert flags == 0


def test_evict_many_sequences_at_the_border():
    """Lengths at keep and around it, more heads than the GPU has CTA slots."""
    kl = [63, 64, 65, 66, 1, 0, 128, 300] * 20
    p = Paged([0] * len(kl), kl, 8, 8, 64, 16, HF, seed=108).cuda()
    mass = (torch.rand(len(kl), 8, p.max_pages * 16, generator=torch.Generator().manual_seed(9)) * 4).round().cuda()
    got = evict(p, mass, 64, 7)                                  # whole numbers: ties everywhere
    assert got[3] == 0
    check_evict(p, mass, 64, 7, got)


def test_evict_rows_longer_than_shared_memory():
    p = Paged([0], [20000], 2, 2, 64, 64, BF, seed=109).cuda()
    mass = torch.rand(1, 2, p.max_pages * 64, generator=torch.Generator().manual_seed(10)).cuda()
    got = evict(p, mass, 5000, 100)
    assert got[3] == 0
    check_evict(p, mass, 5000, 100, got)
