"""Error bounds of the attention over 8-bit pages that take nothing from outside
the row: the output's and the weights' roundings as in the other tests, and for each
of a row's n cells a step of 2^-31 of the row's largest product of weight and value
scale, times codes of up to 448.  (The largest product enters at 2^7 or 2^9 at least;
half steps are binary16's, 2^-25, or the last part's, 2^-23: 2^-32 and 2^-32 + 2^-34 of it.)"""
from __future__ import annotations

import numpy as np
import torch

import oracle
from e4m3_helpers import Codes
from paged_helpers import TINY, UNIT, assert_within


def problem(ql, kl, H_q, H_kv, D, dtype, seed=1):
    p = Codes(ql, kl, H_q, H_kv, D, 16, dtype, seed=seed, spread=0)
    if dtype == torch.float16:                                   # (room below binary16's range)
        p.v_scale[p.v_scale != 255] -= 10
    return p


def check_rows(p, out, lse):
    k, v = p.pools()
    q = p.q.double().numpy()
    args = (p.starts.numpy(), p.kl, p.table.numpy(), p.scale)
    o, ls, spread, reach = oracle.paged_attention(q, k, v, *args)
    n, D, u = max(p.kl), p.D, UNIT[p.dtype]
    # weights: scores, their parts of the queries, the exponential and the sum (as in the other tests)
    w = 2 * ((D + 2) * 2.0 ** -23 * reach + reach * 2.0 ** -22) + 2.0 ** -21 + n * 2.0 ** -23
    d = oracle.paged_attention(q - oracle.e4m3_parts(q, 3 if p.dtype == torch.float16 else 2), k, v, *args)[3]
    most = np.repeat(oracle.e4m3_scale(p.v_scale.numpy()) * 448.0, 16, axis=2)[..., None] * np.ones(D)
    owned = np.zeros(most.shape[0], bool)
    owned[[x for row in p.table.tolist() for x in row if 0 <= x < len(owned)]] = True
    most[~owned] = 0.0
    floor = n * 2.0 ** -31 * oracle.paged_attention(q, k, most, *args)[0]
    bound = u * np.abs(o) + (u + 2 * w[..., None]) * (1 + u) * spread + 4 * d[..., None] * spread + floor + TINY[p.dtype]
    assert_within(out[:p.live], o[:p.live], bound[:p.live], "out")
    assert_within(lse[:p.live], ls[:p.live], (w + 2.0 ** -22 * (1 + np.abs(ls)) + 2 * d)[:p.live], "lse")
