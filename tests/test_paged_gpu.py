"""GPU parity of the paged cache's calls against the FP64 oracle: the store with
several position axes, the attention of chunks and single tokens, the weight per
cell, the eviction, and a run of all four as a server makes it."""
import numpy as np
import pytest
import torch

import kv_cached_gqa_rope_gb300 as kv
import oracle
from paged_helpers import JUNK, TINY, UNIT, Paged, assert_within, attention_bounds, bits16

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


# ------------------------------------------------------------------ store
def store(p, positions, axis, theta=10000.0, q=None, k=None, v=None, ws=None):
    ws = kv.new_workspace(kv.paged_rope_kv_store_workspace_size()) if ws is None else ws
    q_out = torch.full((p.N, p.H_q, p.D), 7.0, dtype=p.dtype, device="cuda")
    kv.paged_rope_kv_store_out_(p.d_q if q is None else q, p.d_k if k is None else k, p.d_v if v is None else v,
                                positions, *p.meta, theta, axis, q_out, p.d_k_cache, p.d_v_cache, ws)
    torch.cuda.synchronize()
    return q_out, kv.kvgqa_read_status(ws)


def check_store(p, q_out, positions, axis, theta, skip=()):
    """Every stored value one rounding from the exact one (plus the FP32
    evaluation's 2^-21 of the pair), every other byte as it was."""
    cells = oracle.paged_token_cells(p.starts.numpy(), p.kl)
    pos = positions.cpu().numpy()
    k_ref, v_ref = bits16(p.k_cache).copy(), bits16(p.v_cache).copy()
    k_got, v_got = bits16(p.d_k_cache), bits16(p.d_v_cache)
    k_all = p.d_k_cache.double().cpu().numpy()
    q_rot = oracle.paged_rope(p.q.double().numpy(), pos, axis, theta)
    k_rot = oracle.paged_rope(p.k.double().numpy(), pos, axis, theta)
    q_new = q_out.double().cpu().numpy()

    def bound(ref, x):
        half = x.shape[-1] // 2
        pair = np.abs(x[..., :half]) + np.abs(x[..., half:])
        return UNIT[p.dtype] * np.abs(ref) + 2.0 ** -21 * np.concatenate([pair, pair], -1) + TINY[p.dtype]

    for n, (a, j) in enumerate(cells):
        pid, o = int(p.table[a, j // p.page]), j % p.page
        if n in skip:
            assert np.all(q_new[n] == 7.0)
            continue
        assert_within(q_new[n], q_rot[n], bound(q_rot[n], p.q[n].double().numpy()), f"q of token {n}")
        assert_within(k_all[pid, :, o], k_rot[n], bound(k_rot[n], p.k[n].double().numpy()), f"k of token {n}")
        v_ref[pid, :, o] = bits16(p.v[n])
        k_ref[pid, :, o] = k_got[pid, :, o]
    assert np.all(q_new[len(cells):] == 7.0)                     # rows behind the last sequence
    assert np.array_equal(k_got, k_ref) and np.array_equal(v_got, v_ref)


@pytest.mark.parametrize("H_q,H_kv,D,page,dtype,sections,interleaved", [
    (4, 2, 64, 16, BF, (32,), False), (32, 8, 128, 32, BF, (16, 24, 24), False), (8, 8, 128, 64, HF, (16, 24, 24), True),
    (5, 5, 64, 128, HF, (10, 11, 11), True), (16, 1, 128, 256, BF, (30, 34), False), (6, 2, 64, 16, BF, (8, 8, 8, 8), True)])
def test_store(H_q, H_kv, D, page, dtype, sections, interleaved):
    p = Paged([1, 17, 0, 64, 1, 5], [1, 40, 9, 64, 300, 261], H_q, H_kv, D, page, dtype, seed=D + page, behind=3).cuda()
    axis = kv.rope_axis_of_pair(sections, interleaved)
    g = torch.Generator().manual_seed(3)
    positions = torch.randint(0, 70000, (len(sections), p.N), generator=g, dtype=torch.int32).cuda()
    positions[0, 0] = 0
    positions[-1, 1] = 2 ** 31 - 1
    q_out, flags = store(p, positions, axis, 500000.0)
    assert flags == 0
    check_store(p, q_out, positions, axis, 500000.0)


def test_store_from_a_fused_projection():
    p = Paged([1] * 40, list(range(1, 41)), 32, 8, 128, 16, BF, seed=5).cuda()
    qkv = torch.cat([p.d_q, p.d_k, p.d_v], 1)
    axis = kv.rope_axis_of_pair((16, 24, 24))
    positions = torch.arange(3 * 40, dtype=torch.int32).view(3, 40).cuda()
    q_out, flags = store(p, positions, axis, 10000.0, qkv[:, :32], qkv[:, 32:40], qkv[:, 40:])
    assert flags == 0
    check_store(p, q_out, positions, axis, 10000.0)


def test_store_many_tokens():
    p = Paged([2100, 700], [2500, 700], 8, 2, 128, 64, BF, seed=6).cuda()
    axis = kv.rope_axis_of_pair((64,))
    positions = torch.arange(p.N, dtype=torch.int32).view(1, -1).cuda()
    q_out, flags = store(p, positions, axis)
    assert flags == 0
    check_store(p, q_out, positions, axis, 10000.0)


def test_store_skips_and_flags_bad_metadata():
    axis = kv.rope_axis_of_pair((32,))
    positions = torch.arange(8, dtype=torch.int32).view(1, -1).cuda()

    def fresh():
        return Paged([2, 3, 3], [20, 33, 3], 4, 2, 64, 16, BF, seed=7).cuda()

    p = fresh()
    p.d_table[1, 2] = p.P                                        # cell 32: sequence 1's last token
    q_out, flags = store(p, positions, axis)
    assert flags == kv.FLAG_PAGE_RANGE
    check_store(p, q_out, positions, axis, 10000.0, skip=(4,))
    p = fresh()
    p.d_table[0, 1] = -1
    q_out, flags = store(p, positions, axis)
    assert flags == kv.FLAG_PAGE_RANGE
    check_store(p, q_out, positions, axis, 10000.0, skip=(0, 1))
    p = fresh()
    bad = positions.clone()
    bad[0, 6] = -1
    q_out, flags = store(p, bad, axis)
    assert flags == kv.FLAG_POSITION_RANGE
    check_store(p, q_out, positions, axis, 10000.0, skip=(6,))
    for length in (2, -5, 10 ** 9, -2 ** 31):                    # fewer cells than tokens, or more than the table has
        p = fresh()
        p.d_lengths[1] = length
        q_out, flags = store(p, positions, axis)
        assert flags == kv.FLAG_POSITION_RANGE
        check_store(p, q_out, positions, axis, 10000.0, skip=(2, 3, 4))


# ------------------------------------------------------------------ attention
def attend(p, q=None, lse=True, max_query_len=None, scale=None, out=None, ws=None):
    ws = kv.new_workspace(kv.paged_gqa_attention_workspace_size(p.H_q, p.H_kv, p.D)) if ws is None else ws
    out = torch.full((p.N, p.H_q, p.D), 7.0, dtype=p.dtype, device="cuda") if out is None else out
    lse = torch.full((p.N, p.H_q), 7.0, dtype=torch.float32, device="cuda") if lse else None
    kv.paged_gqa_attention_out_(p.d_q if q is None else q, p.d_k_cache, p.d_v_cache, *p.meta,
                                p.max_query_len if max_query_len is None else max_query_len,
                                p.scale if scale is None else scale, out, lse, ws)
    torch.cuda.synchronize()
    return out, lse, kv.kvgqa_read_status(ws)


def check_attention(p, out, lse, scale=None, rows=None):
    ref = oracle.paged_attention(p.q.double().numpy(), *p.pools(), p.starts.numpy(), p.kl, p.table.numpy(),
                                 p.scale if scale is None else scale)
    b_out, b_lse = attention_bounds(ref, p.dtype, max(p.kl))
    rows = np.arange(p.live) if rows is None else np.asarray(rows)
    assert_within(out.double().cpu().numpy()[rows], ref[0][rows], b_out[rows], "out")
    if lse is not None:
        assert_within(lse.double().cpu().numpy()[rows], ref[1][rows], b_lse[rows], "lse")
        assert torch.all(lse[p.live:] == 7.0)
    assert torch.all(out[p.live:] == 7.0)                        # rows behind the last sequence


CHUNKS = [
    # one token per sequence, short and long, and the empty sequence between
    ([1, 1, 0, 1, 1], [1, 128, 40, 129, 1000], 4, 2, 64, 16, BF),
    ([1], [1], 1, 1, 128, 16, HF),
    ([1], [5000], 8, 1, 128, 64, BF),
    ([1] * 33, [37 * i + 1 for i in range(33)], 8, 2, 128, 32, HF),
    # chunks: one token more and less than tiles and blocks hold
    ([31, 32, 33, 63, 64, 65], [31, 100, 160, 191, 192, 193], 16, 4, 128, 16, BF),
    ([127, 128, 129, 255, 256, 257], [127, 128, 129, 300, 256, 700], 2, 2, 64, 64, HF),
    # a whole prompt, and a chunk over a long prefix
    ([777], [777], 8, 2, 128, 128, BF),
    ([70], [3001], 8, 2, 64, 256, BF),
    # group sizes that are no power of two, and the largest
    ([1, 5, 40], [300, 5, 340], 6, 2, 128, 16, BF),
    ([1, 9, 130], [200, 70, 131], 15, 3, 64, 32, HF),
    ([2, 17, 50], [2, 300, 50], 12, 1, 128, 16, HF),
    ([3, 16, 100], [130, 16, 300], 16, 1, 64, 16, BF),
    # many sequences of every kind
    ([1, 2, 3, 0, 100, 1, 1, 64, 1] * 5, [500, 2, 260, 7, 400, 1, 64, 128, 1025] * 5, 8, 4, 64, 16, BF),
]


@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_attention(case):
    ql, kl, H_q, H_kv, D, page, dtype = CHUNKS[case]
    p = Paged(ql, kl, H_q, H_kv, D, page, dtype, seed=case, behind=case % 3).cuda()
    out, lse, flags = attend(p)
    assert flags == 0
    check_attention(p, out, lse)


def test_attention_more_sequences_than_threads():
    ql = [1 if i % 3 else i % 7 for i in range(900)]
    p = Paged(ql, [q + (i * 5) % 50 for i, q in enumerate(ql)], 2, 1, 64, 16, BF, seed=90).cuda()
    out, lse, flags = attend(p)
    assert flags == 0
    check_attention(p, out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.125, 1.0])
def test_attention_scales(scale):
    p = Paged([1, 20], [150, 290], 4, 2, 64, 16, BF, seed=20).cuda()
    out, lse, flags = attend(p, scale=scale)
    assert flags == 0
    check_attention(p, out, lse, scale=scale)


def test_attention_large_scores():
    """Scores of +-100 and more: the base of the weights has to follow them."""
    p = Paged([3, 1, 40], [800, 333, 40], 8, 2, 128, 32, HF, seed=21, k_scale=12.0).cuda()
    out, lse, flags = attend(p)
    assert flags == 0
    check_attention(p, out, lse)


def test_attention_without_lse_and_into_16_byte_rows():
    p = Paged([1, 37, 2], [90, 260, 2], 4, 2, 64, 16, BF, seed=22).cuda()
    buf = torch.full((p.N * 4 * 64 + 8,), 7.0, dtype=BF, device="cuda")
    out = buf[8:].view(p.N, 4, 64)                               # 16-byte aligned, not 32
    got, _, flags = attend(p, lse=False, out=out)
    assert flags == 0 and torch.all(buf[:8] == 7.0)
    check_attention(p, got, None)
    again, lse, _ = attend(p)
    assert torch.equal(got, again)


def test_attention_equals_the_slot_cache():
    """Pages that lie like a slot cache's rows: the same output as
    cached_gqa_attention_out_ within both calls' roundings."""
    A, L, H_q, H_kv, D, page = 6, 512, 8, 2, 128, 64
    g = torch.Generator().manual_seed(4)
    kc = torch.randn(A, H_kv, L, D, generator=g).to(BF).cuda()
    vc = torch.randn(A, H_kv, L, D, generator=g).to(BF).cuda()
    q = torch.randn(A, H_q, D, generator=g).to(BF).cuda()
    positions = torch.tensor([0, 5, 127, 128, 300, 511], dtype=torch.int32).cuda()
    rows = torch.arange(A, dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    kv.cached_gqa_attention_out_(q, kc, vc, positions, rows, D ** -0.5, out,
                                 kv.new_workspace(kv.cached_gqa_attention_workspace_size(A, H_q, H_kv, D)))
    pool = [x.view(A, H_kv, L // page, page, D).transpose(1, 2).reshape(-1, H_kv, page, D).contiguous() for x in (kc, vc)]
    table = torch.arange(A * L // page, dtype=torch.int32).view(A, -1).cuda()
    starts = torch.arange(A + 1, dtype=torch.int32).cuda()
    got = torch.empty_like(q)
    ws = kv.new_workspace(kv.paged_gqa_attention_workspace_size(H_q, H_kv, D))
    kv.paged_gqa_attention_out_(q, *pool, starts, positions + 1, table, 1, D ** -0.5, got, None, ws)
    assert kv.kvgqa_read_status(ws) == 0
    # each is within one rounding of its weights (2^-8 of sum p|v| <= 4) and of its output of the exact value
    assert (got.float() - out.float()).abs().max().item() <= 2 * (4 + 4) * 2.0 ** -8


def test_attention_skips_and_flags_bad_metadata():
    def fresh():
        return Paged([2, 30, 3, 1], [20, 133, 3, 700], 4, 2, 64, 16, BF, seed=23).cuda()

    others = [0, 1] + list(range(32, 36))
    for length in (29, -1, 10 ** 9):
        p = fresh()
        p.d_lengths[1] = length
        out, lse, flags = attend(p)
        assert flags == kv.FLAG_POSITION_RANGE
        check_attention(p, out, lse, rows=others)
        assert torch.all(out[2:32] == 7.0) and torch.all(lse[2:32] == 7.0)
    p = fresh()
    out, lse, flags = attend(p, max_query_len=29)                # fewer than sequence 1 has
    assert flags == kv.FLAG_POSITION_RANGE
    check_attention(p, out, lse, rows=others)
    assert torch.all(out[2:32] == 7.0) and torch.all(lse[2:32] == 7.0)
    p = fresh()
    p.d_starts[2] = 1                                            # decreasing: sequence 1 has no tokens that make sense
    out, lse, flags = attend(p)
    assert flags == kv.FLAG_POSITION_RANGE
    check_attention(p, out, lse, rows=[0, 1, 35])
    for entry in (p.P, -1, -2 ** 31, 2 ** 31 - 1):
        p = fresh()
        p.d_table[1, 3] = entry
        out, lse, flags = attend(p)
        assert flags == kv.FLAG_PAGE_RANGE
        check_attention(p, out, lse, rows=others)


def test_attention_in_a_replayed_graph():
    """One capture, replayed over new lengths, tables and values in the same
    buffers, behind a store in the same graph; an ordinary call in between uses
    a workspace of its own."""
    H_q, H_kv, D, page = 8, 2, 128, 16
    a = Paged([1, 40, 0, 1], [700, 90, 30, 17], H_q, H_kv, D, page, BF, seed=30, spare=60).cuda()
    b = Paged([20, 1, 20, 1], [20, 1000, 333, 129], H_q, H_kv, D, page, BF, seed=31, spare=40).cuda()
    ws = kv.new_workspace(kv.paged_gqa_attention_workspace_size(H_q, H_kv, D))
    buf = {n: torch.zeros_like(getattr(b, n)) for n in ("d_q", "d_starts", "d_lengths")}
    P = max(a.P, b.P)
    pools = [torch.zeros(P, H_kv, page, D, dtype=BF, device="cuda") for _ in range(2)]
    table = torch.zeros(4, 70, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(buf["d_q"])
    lse = torch.zeros(b.N, H_q, device="cuda")
    assert a.N == b.N

    def fill(p):
        for n, t in buf.items():
            t.copy_(getattr(p, n))
        pools[0][:p.P].copy_(p.d_k_cache)
        pools[1][:p.P].copy_(p.d_v_cache)
        table.fill_(JUNK)
        table[:, :p.max_pages].copy_(p.d_table)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call = kv.prepare_paged_gqa_attention_out_(buf["d_q"], *pools, buf["d_starts"], buf["d_lengths"], table, 40,
                                                   D ** -0.5, out, lse, ws)
        fill(a)
        call()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            call()
    for p in (b, a, b):
        fill(p)
        graph.replay()
        torch.cuda.synchronize()
        ref = oracle.paged_attention(p.q.double().numpy(), *p.pools(), p.starts.numpy(), p.kl, p.table.numpy(), p.scale)
        b_out, b_lse = attention_bounds(ref, BF, max(p.kl))
        assert_within(out, ref[0], b_out, "out")
        assert_within(lse, ref[1], b_lse, "lse")
        direct, _, _ = attend(p)
        assert torch.equal(direct, out)
    assert kv.kvgqa_read_status(ws) == 0


def test_two_attentions_at_once():
    p = Paged([1, 30, 1], [3000, 500, 2000], 8, 2, 128, 32, BF, seed=33).cuda()
    want, want_lse, _ = attend(p)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.zeros_like(want) for _ in streams]
    works = [kv.new_workspace(kv.paged_gqa_attention_workspace_size(8, 2, 128)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, o, w in zip(streams, outs, works):
            kv.paged_gqa_attention_out_(p.d_q, p.d_k_cache, p.d_v_cache, *p.meta, 30, p.scale, o, None, w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, works):
        assert torch.equal(o, want) and kv.kvgqa_read_status(w) == 0


# ------------------------------------------------------------------ mass
def add_mass(p, lse, mass, max_query_len=None, scale=None):
    ws = kv.new_workspace(kv.paged_attention_mass_workspace_size())
    kv.paged_attention_mass_out_(p.d_q, lse, p.d_k_cache, *p.meta,
                                 p.max_query_len if max_query_len is None else max_query_len,
                                 p.scale if scale is None else scale, mass, ws)
    torch.cuda.synchronize()
    return kv.kvgqa_read_status(ws)


def check_mass(p, got, before, lse, reach, scale=None, seqs=None):
    """A weight is off by w (see attention_bounds) and the rounding of the log
    sum to base 2, 2^-22 of its size; a cell adds at most T * G of them to what
    it had, in FP32."""
    ref = oracle.paged_mass(p.q.double().numpy(), lse, *p.pools()[:1], p.starts.numpy(), p.kl, p.table.numpy(),
                            p.scale if scale is None else scale, before.shape[2])
    w = 2 * ((p.D + 4) * 2.0 ** -23 * np.nanmax(reach) + 2.0 ** -22 * (1 + np.nanmax(np.abs(lse)))) + 2.0 ** -21
    cols = p.max_query_len * p.H_q // p.H_kv
    bound = ref * (w + (cols + 2) * 2.0 ** -24) + np.abs(before) * 2.0 ** -23 + 1e-38
    got = got.double().cpu().numpy()
    want = before + ref
    for a in range(p.A) if seqs is None else seqs:
        n = p.kl[a] if p.ql[a] else 0
        if n:
            assert_within(got[a, :, :n], want[a, :, :n], bound[a, :, :n], f"mass of sequence {a}")
        assert np.array_equal(got[a, :, n:], before[a, :, n:])


@pytest.mark.parametrize("case", range(len(CHUNKS)))
def test_mass(case):
    ql, kl, H_q, H_kv, D, page, dtype = CHUNKS[case]
    p = Paged(ql, kl, H_q, H_kv, D, page, dtype, seed=case, behind=case % 3).cuda()
    ref = oracle.paged_attention(p.q.double().numpy(), *p.pools(), p.starts.numpy(), p.kl, p.table.numpy(), p.scale)
    lse = torch.tensor(np.nan_to_num(ref[1]), dtype=torch.float32)
    mass = torch.rand(p.A, H_kv, max(p.kl) + 3, generator=torch.Generator().manual_seed(1))
    got = mass.cuda()
    assert add_mass(p, lse.cuda(), got) == 0
    check_mass(p, got, mass.double().numpy(), lse.double().numpy(), ref[3])
    again = mass.cuda()
    add_mass(p, lse.cuda(), again)
    assert torch.equal(got, again)


def test_mass_sums_to_the_queries():
    """Every query hands out a weight of one per head."""
    p = Paged([1, 50, 300], [900, 400, 300], 8, 2, 64, 32, BF, seed=40).cuda()
    _, lse, _ = attend(p)
    mass = torch.zeros(p.A, 2, max(p.kl), device="cuda")
    assert add_mass(p, lse, mass) == 0
    total = mass.double().sum(2).cpu().numpy()
    assert np.allclose(total, np.array(p.ql)[:, None] * 4.0, rtol=2e-5, atol=0)


def test_mass_skips_and_flags_bad_metadata():
    def fresh():
        return Paged([2, 30, 3], [20, 133, 300], 4, 2, 64, 16, BF, seed=41).cuda()

    p = fresh()
    ref = oracle.paged_attention(p.q.double().numpy(), *p.pools(), p.starts.numpy(), p.kl, p.table.numpy(), p.scale)
    lse = torch.tensor(ref[1], dtype=torch.float32)
    before = np.ones((3, 2, 320))
    args = (before, lse.double().numpy(), ref[3])
    for length in (29, 10 ** 9):
        p = fresh()
        p.d_lengths[1] = length
        mass = torch.ones(3, 2, 320, device="cuda")
        assert add_mass(p, lse.cuda(), mass) == kv.FLAG_POSITION_RANGE
        check_mass(p, mass, *args, seqs=[0, 2])
        assert torch.all(mass[1] == 1)
    p = fresh()
    mass = torch.ones(3, 2, 200, device="cuda")                  # fewer cells than sequence 2 has
    assert add_mass(p, lse.cuda(), mass) == kv.FLAG_POSITION_RANGE
    assert torch.all(mass[2] == 1)
    wide = torch.ones(3, 2, 320, device="cuda")
    assert add_mass(p, lse.cuda(), wide) == 0
    check_mass(p, wide, *args)
    assert torch.equal(mass[:2], wide[:2, :, :200])
    p = fresh()
    p.d_table[1, 3] = p.P
    mass = torch.ones(3, 2, 320, device="cuda")
    assert add_mass(p, lse.cuda(), mass) == kv.FLAG_PAGE_RANGE
    check_mass(p, mass, *args, seqs=[0, 2])


# ------------------------------------------------------------------ eviction
def evict(p, mass, keep, recent):
    A, H_kv, M = mass.shape
    ws = kv.new_workspace(kv.paged_evict_workspace_size(A, H_kv, keep))
    mass_out = torch.full((A, H_kv, M), 7.0, device="cuda")
    kept = torch.full((A, H_kv, keep), 7, dtype=torch.int32, device="cuda")
    lengths = torch.full((A,), 7, dtype=torch.int32, device="cuda")
    kv.paged_evict_out_(mass, p.d_lengths, p.d_table, keep, recent, p.d_k_cache, p.d_v_cache, mass_out, kept, lengths, ws)
    torch.cuda.synchronize()
    return mass_out, kept, lengths, kv.kvgqa_read_status(ws)


def check_evict(p, mass, keep, recent, got, seqs=None):
    mass_out, kept, lengths, _ = got
    k, v, m_ref, k_ref, n_ref = oracle.paged_evict(mass.cpu().numpy(), p.kl, p.table.numpy(), keep, recent,
                                                   bits16(p.k_cache), bits16(p.v_cache))
    seqs = range(p.A) if seqs is None else seqs
    for a in seqs:
        assert np.array_equal(kept[a].cpu().numpy(), k_ref[a])
        assert np.array_equal(mass_out[a].cpu().numpy(), m_ref[a], equal_nan=True)
        assert int(lengths[a]) == n_ref[a]
    if len(seqs) == p.A:
        assert np.array_equal(bits16(p.d_k_cache), k) and np.array_equal(bits16(p.d_v_cache), v)


@pytest.mark.parametrize("kl,H_kv,D,page,dtype,keep,recent", [
    ([1, 2, 3, 40, 300], 2, 64, 16, BF, 2, 1), ([1000, 64, 65, 0, 127], 3, 128, 16, HF, 64, 0),
    ([5000], 1, 128, 64, BF, 1000, 100), ([700, 701, 900], 8, 64, 256, HF, 700, 700),
    ([33, 5], 2, 128, 32, BF, 1, 0), ([2100] * 5, 4, 128, 128, BF, 2099, 3), ([50, 60], 2, 64, 16, BF, 500, 20)])
def test_evict(kl, H_kv, D, page, dtype, keep, recent):
    p = Paged([0] * len(kl), kl, H_kv, H_kv, D, page, dtype, seed=keep).cuda()
    M = p.max_pages * page
    mass = torch.rand(p.A, H_kv, M, generator=torch.Generator().manual_seed(2)) ** 6
    mass = mass.cuda()
    got = evict(p, mass, keep, recent)
    assert got[3] == 0
    check_evict(p, mass, keep, recent, got)


def test_evict_ties_and_strange_masses():
    """Equal masses go to the lowest cell; -0 equals 0; infinities are the
    extremes and NaN comes after everything."""
    p = Paged([0] * 4, [600, 601, 640, 333], 2, 2, 64, 16, BF, seed=50).cuda()
    g = torch.Generator().manual_seed(3)
    choice = torch.tensor([0.0, -0.0, 1.0, 1.0000001, -1.0, float("inf"), float("-inf"), float("nan"), 1e-45, 3e38])
    mass = choice[torch.randint(0, 10, (4, 2, 656), generator=g)].cuda()
    mass[1] = 0.0
    mass[3] = float("nan")
    for keep, recent in ((1, 0), (64, 10), (300, 0), (332, 331), (599, 64)):
        q = Paged([0] * 4, [600, 601, 640, 333], 2, 2, 64, 16, BF, seed=50).cuda()
        got = evict(q, mass, keep, recent)
        assert got[3] == 0
        check_evict(q, mass, keep, recent, got)


def test_evict_skips_and_flags_bad_metadata():
    def fresh():
        return Paged([0] * 3, [100, 200, 300], 2, 2, 64, 16, BF, seed=51).cuda()

    mass = torch.rand(3, 2, 320, device="cuda")
    p = fresh()
    p.d_table[1, 12] = p.P                                       # needed: a kept cell may lie there
    got = evict(p, mass, 64, 8)
    assert got[3] == kv.FLAG_PAGE_RANGE
    check_evict(p, mass, 64, 8, got, seqs=[0, 2])
    assert torch.all(got[1][1] == 7) and int(got[2][1]) == 7 and torch.all(got[0][1] == 7)
    rows = p.table[1, :13].long()
    assert np.array_equal(bits16(p.d_k_cache[rows.cuda()]), bits16(p.k_cache[rows]))
    for length in (-1, 10 ** 9):
        p = fresh()
        p.d_lengths[1] = length
        got = evict(p, mass, 64, 8)
        assert got[3] == kv.FLAG_POSITION_RANGE
        check_evict(p, mass, 64, 8, got, seqs=[0, 2])
        assert torch.all(got[1][1] == 7) and int(got[2][1]) == 7
    p = fresh()
    got = evict(p, mass[:, :, :250].contiguous(), 64, 8)         # fewer cells than sequence 2 has
    assert got[3] == kv.FLAG_POSITION_RANGE
    assert torch.all(got[1][2] == 7) and int(got[2][2]) == 7 and torch.all(got[0][2] == 7)
    whole = evict(fresh(), mass, 64, 8)
    assert whole[3] == 0
    assert torch.equal(got[1][:2], whole[1][:2]) and torch.equal(got[0][:2], whole[0][:2, :, :250])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", [BF, HF])
def test_a_server_s_steps(dtype):
    """A prompt in two chunks, decode steps with their weights added up, an
    eviction, and decode steps on what is left; the oracle keeps its own state
    from what the library stored, step by step."""
    H_q, H_kv, D, page, A, theta = 8, 2, 64, 16, 3, 10000.0
    g = torch.Generator().manual_seed(60)
    max_pages, P = 14, 40
    pools = [torch.full((P, H_kv, page, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    table = torch.randperm(P, generator=g)[:A * 13].view(A, 13).to(torch.int32)
    table = torch.cat([table, torch.full((A, 1), JUNK, dtype=torch.int32)], 1).cuda()
    assert table.shape == (A, max_pages)
    M = max_pages * page
    mass = torch.zeros(A, H_kv, M, device="cuda")
    axis = kv.rope_axis_of_pair((8, 12, 12))
    ws_s = kv.new_workspace(kv.paged_rope_kv_store_workspace_size())
    ws_a = kv.new_workspace(kv.paged_gqa_attention_workspace_size(H_q, H_kv, D))
    ws_m = kv.new_workspace(kv.paged_attention_mass_workspace_size())
    lengths = [0] * A
    position = [0] * A

    def step(ql):
        nonlocal lengths
        N = sum(ql)
        q, k, v = (torch.randn(N, h, D, generator=g).to(dtype) for h in (H_q, H_kv, H_kv))
        starts = np.concatenate([[0], np.cumsum(ql)])
        lengths = [n + x for n, x in zip(lengths, ql)]
        pos = np.concatenate([np.arange(position[a], position[a] + ql[a]) for a in range(A)])
        for a in range(A):
            position[a] += ql[a]
        pos = np.stack([pos, pos + 1, pos * 2])
        d = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        meta = (d(starts), d(lengths), table)
        q_rot, out = torch.empty_like(q, device="cuda"), torch.empty_like(q, device="cuda")
        lse = torch.empty(N, H_q, device="cuda")
        kv.paged_rope_kv_store_out_(q.cuda(), k.cuda(), v.cuda(), d(pos), *meta, theta, axis, q_rot, *pools, ws_s)
        kv.paged_gqa_attention_out_(q_rot, *pools, *meta, max(ql), D ** -0.5, out, lse, ws_a)
        before = mass.double().cpu().numpy()
        kv.paged_attention_mass_out_(q_rot, lse, pools[0], *meta, max(ql), D ** -0.5, mass, ws_m)
        torch.cuda.synchronize()
        rot = oracle.paged_rope(q.double().numpy(), pos, axis, theta)
        assert np.abs(q_rot.double().cpu().numpy() - rot).max() <= UNIT[dtype] * (np.abs(rot).max() + 1)
        host = [np.nan_to_num(x.double().cpu().numpy()) for x in pools]
        tb = table.cpu().numpy()
        ref = oracle.paged_attention(q_rot.double().cpu().numpy(), *host, starts, lengths, tb, D ** -0.5)
        b_out, b_lse = attention_bounds(ref, dtype, max(lengths))
        assert_within(out, ref[0], b_out, "out")
        assert_within(lse, ref[1], b_lse, "lse")
        add = oracle.paged_mass(q_rot.double().cpu().numpy(), lse.double().cpu().numpy(), host[0], starts, lengths, tb,
                                D ** -0.5, M)
        assert np.abs(mass.double().cpu().numpy() - before - add).max() <= 1e-4 * (1 + add.max())

    step([100, 37, 1])
    step([63, 90, 2])
    for _ in range(5):
        step([1, 1, 1])
    keep, recent = 48, 16
    ws_e = kv.new_workspace(kv.paged_evict_workspace_size(A, H_kv, keep))
    mass_out = torch.empty_like(mass)
    kept = torch.empty(A, H_kv, keep, dtype=torch.int32, device="cuda")
    new = torch.empty(A, dtype=torch.int32, device="cuda")
    want = oracle.paged_evict(mass.cpu().numpy(), lengths, table.cpu().numpy(), keep, recent, bits16(pools[0]), bits16(pools[1]))
    kv.paged_evict_out_(mass, torch.tensor(lengths, dtype=torch.int32).cuda(), table, keep, recent, *pools, mass_out, kept, new, ws_e)
    torch.cuda.synchronize()
    assert np.array_equal(bits16(pools[0]), want[0]) and np.array_equal(bits16(pools[1]), want[1])
    assert np.array_equal(kept.cpu().numpy(), want[3]) and new.tolist() == want[4].tolist()
    mass.copy_(mass_out)
    lengths = new.tolist()
    assert lengths == [48, 48, 8]
    for a in range(A):                                           # the freed pages are someone else's now
        table[a, -(-(lengths[a] + 4) // page):] = JUNK
    for _ in range(4):
        step([1, 1, 1])
    assert [kv.kvgqa_read_status(w) for w in (ws_s, ws_a, ws_m, ws_e)] == [0, 0, 0, 0]
