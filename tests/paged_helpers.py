"""A seeded paged cache with packed new tokens, on the host and on the GPU, and
the error bounds of the tests on it."""
from __future__ import annotations

import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}  # the smallest subnormal
JUNK = 1 << 30  # a block_table entry nothing may use


class Paged:
    """A sequences with ql[a] new tokens among kl[a] cells; the pages in any
    order, everything that no sequence owns set to NaN, table entries behind a
    sequence's last page to JUNK; `behind` rows of the packed tensors belong to
    no sequence."""

    def __init__(self, ql, kl, H_q, H_kv, D, page, dtype=torch.bfloat16, seed=0, behind=0, k_scale=1.0, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.ql, self.kl, self.dtype = list(ql), list(kl), dtype
        self.A, self.H_q, self.H_kv, self.D, self.page = len(self.ql), H_q, H_kv, D, page
        self.N = sum(self.ql) + behind
        need = [-(-n // page) for n in self.kl]
        self.max_pages = max(need, default=0) + 1
        self.P = sum(need) + spare
        ids = torch.randperm(self.P, generator=g).tolist()
        self.table = torch.full((self.A, self.max_pages), JUNK, dtype=torch.int32)
        at = 0
        nan = float("nan")
        self.k_cache = torch.full((self.P, H_kv, page, D), nan, dtype=dtype)
        self.v_cache = torch.full((self.P, H_kv, page, D), nan, dtype=dtype)
        for a, n in enumerate(self.kl):
            for i in range(need[a]):
                pid, cells = ids[at], min(page, n - i * page)
                at += 1
                self.table[a, i] = pid
                self.k_cache[pid, :, :cells] = (torch.randn(H_kv, cells, D, generator=g) * k_scale).to(dtype)
                self.v_cache[pid, :, :cells] = torch.randn(H_kv, cells, D, generator=g).to(dtype)
        self.starts = torch.tensor(np.concatenate([[0], np.cumsum(self.ql)]), dtype=torch.int32)
        self.lengths = torch.tensor(self.kl, dtype=torch.int32)
        self.q = torch.randn(self.N, H_q, D, generator=g).to(dtype)
        self.k = torch.randn(self.N, H_kv, D, generator=g).to(dtype)
        self.v = torch.randn(self.N, H_kv, D, generator=g).to(dtype)
        self.scale = D ** -0.5
        self.max_query_len = max(self.ql, default=0)
        self.live = sum(self.ql)

    def cuda(self):
        for name in ("table", "k_cache", "v_cache", "starts", "lengths", "q", "k", "v"):
            setattr(self, "d_" + name, getattr(self, name).cuda())
        return self

    @property
    def meta(self):
        return self.d_starts, self.d_lengths, self.d_table

    def pools(self):
        """The pools as float64 (cells of no sequence as zeros)."""
        return [np.nan_to_num(x.double().numpy(), nan=0.0) for x in (self.k_cache, self.v_cache)]


def bits16(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy()


def attention_bounds(ref, dtype, n):
    """Elementwise error bounds of (out, lse) against the FP64 attention.

    A score is a sum of D products accumulated in FP32 with at most one unit
    (2^-23) lost per addition: off by d = (D + 2) 2^-23 reach at most, and the
    FP32 scaling and the base-2 exponential by 2^-21 of a weight more (the
    scaled score, at most reach log2 e in size, is rounded once).  A weight is
    then off by w = 2 (d + reach 2^-22) + 2^-21 relative to the true one (first
    order, doubled), the sum of n weights by n 2^-24 more.  The weight that
    enters the second product is rounded to the storage type (u; below the
    normal range of binary16 by half its smallest step 2^-25, with the largest
    weight of a row at least 1), the n products are accumulated in FP32 (n
    2^-23), and the output is rounded once more (u).  The sum l in the
    denominator is of the unrounded weights.
    """
    out, lse, spread, reach = ref
    D = out.shape[-1]
    u = UNIT[dtype]
    w = 2 * ((D + 2) * 2.0 ** -23 * reach + reach * 2.0 ** -22) + 2.0 ** -21 + n * 2.0 ** -23
    b_out = u * np.abs(out) + (u + 2 * w[..., None]) * (1 + u) * spread + TINY[dtype]
    if dtype == torch.float16:
        b_out = b_out + n * 2.0 ** -25 * 6.0  # |v| < 6 in these draws' bulk
    b_lse = w + 2.0 ** -22 * (1 + np.abs(lse))
    return b_out, b_lse


def assert_within(got, ref, bound, what):
    got = got.detach().double().cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert np.all(np.isfinite(got)), f"{what}: non-finite values"
    over = np.abs(got - ref) / bound
    assert over.max() <= 1.0, f"{what}: {int((over > 1).sum())} values beyond their bound (worst {over.max():.2f} times)"
