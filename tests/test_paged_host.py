"""Host-side contract of the paged cache's calls, without a GPU: malformed
calls are rejected with the documented status before CUDA is touched, and the
oracle's paged definitions agree with its slot-cache ones and with closed
forms."""
import numpy as np
import pytest
import torch

import kv_cached_gqa_rope_gb300 as kv
import oracle
from paged_helpers import Paged, bits16

BF, HF, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
PAST_THE_CHECKS = ("ECUDA", "EDEVICE")  # a legal call gets this far without a GPU


def aligned_bytes(n):
    raw = torch.zeros(n + 256, dtype=torch.uint8)
    off = (-raw.data_ptr()) % 256
    return raw[off:off + n]


def code_of(fn, **kw):
    if torch.cuda.is_available():
        pytest.skip("host tensors on a GPU box")
    with pytest.raises(kv.KvgqaError) as e:
        fn(**kw)
    return e.value.code


def meta(A=2, N=3, max_pages=2):
    return dict(query_starts=torch.tensor([0, 1, 3], dtype=I32)[:A + 1], kv_lengths=torch.full((A,), 20, dtype=I32),
                block_table=torch.zeros(A, max_pages, dtype=I32))


def caches(P=4, H_kv=2, page=16, D=64, dtype=BF):
    return dict(k_cache=torch.zeros(P, H_kv, page, D, dtype=dtype), v_cache=torch.zeros(P, H_kv, page, D, dtype=dtype))


def store_args(N=3, H_q=4, H_kv=2, D=64, **kw):
    a = dict(q=torch.zeros(N, H_q, D, dtype=BF), k=torch.zeros(N, H_kv, D, dtype=BF), v=torch.zeros(N, H_kv, D, dtype=BF),
             positions=torch.zeros(3, N, dtype=I32), theta=1e4, axis_of_pair=[0] * (D // 2),
             q_out=torch.zeros(N, H_q, D, dtype=BF), workspace=aligned_bytes(256), **meta(), **caches(H_kv=H_kv, D=D))
    a.update(kw)
    return a


def attention_args(N=3, H_q=4, H_kv=2, D=64, **kw):
    a = dict(q_rot=torch.zeros(N, H_q, D, dtype=BF), max_query_len=2, scale=0.125, out=torch.zeros(N, H_q, D, dtype=BF),
             lse=torch.zeros(N, H_q), workspace=aligned_bytes(256), **meta(), **caches(H_kv=H_kv, D=D))
    a.update(kw)
    return a


def mass_args(N=3, H_q=4, H_kv=2, D=64, **kw):
    a = dict(q_rot=torch.zeros(N, H_q, D, dtype=BF), lse=torch.zeros(N, H_q), max_query_len=2, scale=0.125,
             mass=torch.zeros(2, H_kv, 32), workspace=aligned_bytes(256), **meta(),
             k_cache=torch.zeros(4, H_kv, 16, D, dtype=BF))
    a.update(kw)
    return a


def evict_args(H_kv=2, D=64, keep=8, **kw):
    m = meta()
    m.pop("query_starts")
    a = dict(mass=torch.zeros(2, H_kv, 32), keep=keep, recent=2, mass_out=torch.zeros(2, H_kv, 32),
             kept=torch.zeros(2, H_kv, keep, dtype=I32), new_lengths=torch.zeros(2, dtype=I32),
             workspace=aligned_bytes(256), **m, **caches(H_kv=H_kv, D=D))
    a.update(kw)
    return a


CALLS = [(kv.paged_rope_kv_store_out_, store_args), (kv.paged_gqa_attention_out_, attention_args),
         (kv.paged_attention_mass_out_, mass_args), (kv.paged_evict_out_, evict_args)]


@pytest.mark.parametrize("fn,args", CALLS)
def test_legal_calls_get_past_the_checks(fn, args):
    assert code_of(fn, **args()) in PAST_THE_CHECKS


@pytest.mark.parametrize("fn,args", CALLS)
def test_shared_refusals(fn, args):
    a = args()
    assert code_of(fn, **args(kv_lengths=torch.zeros(2, dtype=torch.uint8))) == "EDTYPE"
    assert code_of(fn, **args(kv_lengths=torch.zeros(2, 1, dtype=I32))) == "EINVAL"
    assert code_of(fn, **args(block_table=torch.zeros(3, 2, dtype=I32))) == "EINVAL"
    assert code_of(fn, **args(block_table=torch.zeros(2, 2, dtype=I32).T)) == "ELAYOUT"
    assert code_of(fn, **args(block_table=torch.zeros(2, dtype=I32))) == "EINVAL"
    if "query_starts" in a:
        assert code_of(fn, **args(query_starts=torch.zeros(2, dtype=I32))) == "EINVAL"
    assert code_of(fn, **args(k_cache=torch.zeros(4, 2, 16, 64, dtype=F32))) == "EDTYPE"
    wrong = torch.zeros(4, 2, 16, 64, dtype=HF)
    if fn is not kv.paged_evict_out_:                             # there k_cache names the type
        assert code_of(fn, **args(k_cache=wrong)) == "EDTYPE"
    if "v_cache" in a:
        assert code_of(fn, **args(v_cache=wrong)) == "EDTYPE"
        assert code_of(fn, **args(v_cache=torch.zeros(4, 2, 32, 64, dtype=BF))) == "EINVAL"
        assert code_of(fn, **args(v_cache=a["k_cache"], k_cache=a["k_cache"])) in ("EALIAS",) + PAST_THE_CHECKS
    if fn is not kv.paged_evict_out_:                             # there k_cache names the width
        assert code_of(fn, **args(k_cache=torch.zeros(4, 2, 16, 128, dtype=BF))) == "EINVAL"
        assert code_of(fn, **args(k_cache=torch.zeros(4, 3, 16, 64, dtype=BF))) == "EINVAL"
    for page, code in ((8, "EUNSUPPORTED"), (24, "EUNSUPPORTED"), (512, "EUNSUPPORTED")):
        c = {n: torch.zeros(4, 2, page, 64, dtype=BF) for n in ("k_cache", "v_cache") if n in a}
        assert code_of(fn, **args(**c)) == code
    assert code_of(fn, **args(workspace=torch.zeros(4, dtype=torch.uint8))) == "EWORKSPACE"
    assert code_of(fn, **args(workspace=torch.zeros(64, dtype=I32))) == "EWORKSPACE"


@pytest.mark.parametrize("fn,args", CALLS)
def test_pools_past_the_kernels_indexes_are_refused(fn, args, monkeypatch):
    # 2^26 pages of 2 heads and 256 cells: 2^32 groups of 8 rows (no such memory
    # exists; the descriptors say so)
    plain = kv.describe

    def described(t):
        d = plain(t)
        if t.dim() == 4:
            d.shape[0], d.shape[2], d.bytes = 1 << 26, 256, 1 << 62
            d.strides[0], d.strides[1] = 2 * 256 * 64, 256 * 64
        return d

    monkeypatch.setattr(kv, "describe", described)
    assert code_of(fn, **args()) == "EUNSUPPORTED"


def test_store_refusals():
    fn = kv.paged_rope_kv_store_out_
    assert code_of(fn, **store_args(theta=0.0)) == "EINVAL"
    assert code_of(fn, **store_args(positions=torch.zeros(3, 4, dtype=I32))) == "EINVAL"
    assert code_of(fn, **store_args(positions=torch.zeros(5, 3, dtype=I32))) == "EINVAL"
    assert code_of(fn, **store_args(positions=torch.zeros(0, 3, dtype=I32))) == "EINVAL"
    assert code_of(fn, **store_args(positions=torch.zeros(3, dtype=I32))) == "EINVAL"
    assert code_of(fn, **store_args(axis_of_pair=[0] * 31 + [3])) == "EINVAL"
    with pytest.raises(ValueError):
        fn(**store_args(axis_of_pair=[0] * 31))
    with pytest.raises(ValueError):
        fn(**store_args(axis_of_pair=[0] * 31 + [-1]))
    assert code_of(fn, **store_args(k=torch.zeros(3, 1, 64, dtype=BF))) == "EINVAL"
    assert code_of(fn, **store_args(q_out=torch.zeros(3, 4, 64, dtype=HF))) == "EDTYPE"
    qkv = torch.zeros(3, 8, 64, dtype=BF)                         # views of a fused projection are taken
    assert code_of(fn, **store_args(q=qkv[:, :4], k=qkv[:, 4:6], v=qkv[:, 6:])) in PAST_THE_CHECKS
    odd = torch.zeros(3, 4 * 64 + 4, dtype=BF)[:, :256].view(3, 4, 64)
    assert code_of(fn, **store_args(q=odd)) == "ELAYOUT"          # rows not a multiple of 16 bytes apart
    assert code_of(fn, **store_args(q=torch.zeros(3, 64, 4, dtype=BF).transpose(1, 2))) == "ELAYOUT"
    assert code_of(fn, **store_args(q=torch.zeros(1, 4, 64, dtype=BF).expand(3, 4, 64))) == "ELAYOUT"
    assert code_of(fn, **store_args(q=torch.zeros(3 * 256 + 1, dtype=BF)[1:].view(3, 4, 64))) == "ELAYOUT"
    a = store_args()
    assert code_of(fn, **dict(a, q_out=a["q"])) == "EALIAS"
    assert code_of(fn, **store_args(D=32)) == "EUNSUPPORTED"
    assert code_of(fn, **store_args(H_q=3)) == "EINVAL"


def test_attention_refusals():
    fn = kv.paged_gqa_attention_out_
    assert code_of(fn, **attention_args(lse=None)) in PAST_THE_CHECKS
    assert code_of(fn, **attention_args(lse=torch.zeros(3, 4, dtype=BF))) == "EDTYPE"
    assert code_of(fn, **attention_args(lse=torch.zeros(3, 2))) == "EINVAL"
    assert code_of(fn, **attention_args(scale=float("nan"))) == "EINVAL"
    assert code_of(fn, **attention_args(max_query_len=-1)) == "EINVAL"
    assert code_of(fn, **attention_args(H_q=34)) == "EUNSUPPORTED"    # 17 heads to a group
    assert code_of(fn, **attention_args(out=torch.zeros(4, 4, 64, dtype=BF))) == "EINVAL"
    a = attention_args()
    assert code_of(fn, **dict(a, out=a["q_rot"])) == "EALIAS"
    assert code_of(fn, **attention_args(block_table=torch.zeros(2, 1, dtype=I32).expand(2, 1 << 27))) in ("ELAYOUT", "EUNSUPPORTED")
    with pytest.raises(kv.KvgqaError) as e:
        kv.paged_gqa_attention_workspace_size(4, 2, 96, 0)
    assert e.value.code == "EUNSUPPORTED"
    with pytest.raises(kv.KvgqaError) as e:
        kv.paged_gqa_attention_workspace_size(5, 2, 64, 0)
    assert e.value.code == "EINVAL"


def test_mass_refusals():
    fn = kv.paged_attention_mass_out_
    assert code_of(fn, **mass_args(mass=torch.zeros(2, 2, 32, dtype=BF))) == "EDTYPE"
    assert code_of(fn, **mass_args(mass=torch.zeros(3, 2, 32))) == "EINVAL"
    assert code_of(fn, **mass_args(mass=torch.zeros(2, 32, 2).transpose(1, 2))) == "ELAYOUT"
    assert code_of(fn, **mass_args(lse=torch.zeros(3, 4, dtype=HF))) == "EDTYPE"
    assert code_of(fn, **mass_args(scale=float("inf"))) == "EINVAL"
    both = torch.zeros(2, 2, 32)
    assert code_of(fn, **mass_args(mass=both, lse=both.view(-1)[:12].view(3, 4))) == "EALIAS"


def test_evict_refusals():
    fn = kv.paged_evict_out_
    for keep, recent in ((0, 0), (-1, 0), (8, 9), (8, -1)):
        assert code_of(fn, **dict(evict_args(), keep=keep, recent=recent)) == "EINVAL"
    assert code_of(fn, **evict_args(kept=torch.zeros(2, 2, 9, dtype=I32))) == "EINVAL"
    assert code_of(fn, **evict_args(kept=torch.zeros(2, 2, 8))) == "EDTYPE"
    assert code_of(fn, **evict_args(new_lengths=torch.zeros(3, dtype=I32))) == "EINVAL"
    assert code_of(fn, **evict_args(mass_out=torch.zeros(2, 2, 31))) == "EINVAL"
    a = evict_args()
    assert code_of(fn, **dict(a, mass_out=a["mass"])) == "EALIAS"
    assert code_of(fn, **dict(a, new_lengths=a["kv_lengths"])) == "EALIAS"
    assert code_of(fn, **evict_args(D=96)) == "EUNSUPPORTED"
    for bad in ((-1, 1, 1), (1, 0, 1), (1, 1, 0)):
        with pytest.raises(kv.KvgqaError) as e:
            kv.paged_evict_workspace_size(*bad)
        assert e.value.code == "EINVAL"


def test_empty_operands_of_any_stride_are_taken():
    """A call without tokens, as torch strides its tensors."""
    m = dict(query_starts=torch.zeros(3, dtype=I32), kv_lengths=torch.full((2,), 20, dtype=I32),
             block_table=torch.zeros(2, 2, dtype=I32))
    assert code_of(kv.paged_rope_kv_store_out_, **dict(store_args(N=0), **m)) in PAST_THE_CHECKS
    assert code_of(kv.paged_gqa_attention_out_, **dict(attention_args(N=0), **m)) in PAST_THE_CHECKS
    assert code_of(kv.paged_attention_mass_out_, **dict(mass_args(N=0), **m)) in PAST_THE_CHECKS
    m["block_table"] = torch.zeros(2, 0, dtype=I32)               # and a table without pages
    assert code_of(kv.paged_attention_mass_out_, **dict(mass_args(N=0), **m)) in PAST_THE_CHECKS
    a = evict_args(mass=torch.zeros(2, 2, 0), mass_out=torch.zeros(2, 2, 0), block_table=m["block_table"])
    assert code_of(kv.paged_evict_out_, **a) in PAST_THE_CHECKS


def test_workspace_sizes():
    assert kv.paged_rope_kv_store_workspace_size() == 256
    assert kv.paged_attention_mass_workspace_size() == 256
    assert kv.paged_evict_workspace_size(4, 8, 100) == 256


def test_axis_of_pair():
    assert kv.rope_axis_of_pair((2, 3)) == [0, 0, 1, 1, 1]
    assert kv.rope_axis_of_pair((2, 4, 1), interleaved=True) == [0, 1, 2, 0, 1, 1, 1]
    assert kv.rope_axis_of_pair((32,)) == [0] * 32
    with pytest.raises(ValueError):
        kv.rope_axis_of_pair(())
    with pytest.raises(ValueError):
        kv.rope_axis_of_pair((3, -1))


# ------------------------------------------------------------------ the oracle
def test_oracle_attention_agrees_with_the_slot_cache():
    p = Paged([1, 1, 1], [5, 17, 64], 4, 2, 64, 16, seed=1)
    out, lse, spread, reach = oracle.paged_attention(p.q.double().numpy(), *p.pools(), p.starts.numpy(), p.kl,
                                                     p.table.numpy(), p.scale)
    kc = np.zeros((3, 2, 64, 64), dtype=np.uint16)
    vc = np.zeros_like(kc)
    for a, n in enumerate(p.kl):
        kc[a, :, :n] = oracle.paged_cells(bits16(p.k_cache).view(np.uint16), p.table[a].numpy(), n)
        vc[a, :, :n] = oracle.paged_cells(bits16(p.v_cache).view(np.uint16), p.table[a].numpy(), n)
    ref = oracle.cached_gqa_attention(bits16(p.q).view(np.uint16), kc, vc, np.array(p.kl) - 1, np.arange(3), p.scale)
    assert np.allclose(out, ref, rtol=1e-12, atol=1e-12)
    assert np.all(spread >= np.abs(out)) and np.all(reach > 0)
    # the weights sum to one per query head
    mass = oracle.paged_mass(p.q.double().numpy(), lse, p.pools()[0], p.starts.numpy(), p.kl, p.table.numpy(), p.scale, 70)
    assert np.allclose(mass.sum(2), 2.0, rtol=1e-12)


def test_oracle_chunk_equals_its_tokens_one_by_one():
    p = Paged([7], [20], 2, 1, 64, 16, seed=2)
    args = (*p.pools(),)
    out, lse, _, _ = oracle.paged_attention(p.q.double().numpy(), *args, p.starts.numpy(), p.kl, p.table.numpy(), p.scale)
    for t in range(7):
        o, l, _, _ = oracle.paged_attention(p.q[t:t + 1].double().numpy(), *args, [0, 1], [14 + t], p.table.numpy(), p.scale)
        assert np.allclose(out[t], o[0]) and np.allclose(lse[t], l[0])


def test_oracle_rope_agrees_on_one_axis():
    g = np.random.default_rng(0)
    x, pos = g.standard_normal((5, 3, 64)), g.integers(0, 9000, (1, 5))
    assert np.allclose(oracle.paged_rope(x, pos, [0] * 32, 5e5), oracle.rope_split_half(x, pos[0][:, None], 5e5), atol=1e-12)
    axis = [0, 1] * 16                                            # and pair by pair on two
    two = oracle.paged_rope(x, np.stack([pos[0], pos[0] + 7]), axis, 5e5)
    other = oracle.rope_split_half(x, pos[0][:, None] + 7, 5e5)
    assert np.allclose(two[..., 1::2], other[..., 1::2], atol=1e-12)


def test_oracle_evict_by_hand():
    p = Paged([0], [6], 1, 1, 64, 16, seed=3)
    mass = np.array([[[0.5, 2.0, 0.5, np.nan, 0.1, 0.0, 9.0]]])
    k, v, m, kept, n = oracle.paged_evict(mass, p.kl, p.table.numpy(), 3, 1, *p.pools())
    assert kept.tolist() == [[[0, 1, 5]]] and m[0, 0].tolist() == [0.5, 2.0, 0.0, 0, 0, 0, 0] and n.tolist() == [3]
    pid = int(p.table[0, 0])
    assert np.array_equal(k[pid, 0, 2], p.pools()[0][pid, 0, 5]) and np.array_equal(v[pid, 0, 1], p.pools()[1][pid, 0, 1])
