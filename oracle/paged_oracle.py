"""FP64 definitions of the paged cache's operations, as plain loops over
sequences in numpy.

TEST INFRASTRUCTURE, like the rest of this package.  Values come in and go out
as float64 arrays (nothing is rounded here; tests bound the rounding), metadata
as integers:

  k_pool, v_pool [P, H_kv, page, D]; block_table [A, max_pages]; query_starts
  [A + 1]; kv_lengths [A].  Cell j of sequence a is cell j % page of page
  block_table[a, j // page]; its new tokens, rows query_starts[a] .. of the
  packed tensors, are its last cells, and a token sees the cells up to its own.
"""
from __future__ import annotations

import numpy as np

__all__ = ["paged_cells", "paged_token_cells", "paged_rope", "paged_attention", "paged_mass", "paged_evict"]


def paged_cells(pool, table_row, n):
    """A sequence's first n cells in order, [H_kv, n, D]."""
    page = pool.shape[2]
    j = np.arange(n)
    return pool[np.asarray(table_row)[j // page], :, j % page].transpose(1, 0, 2)


def paged_token_cells(query_starts, kv_lengths):
    """(sequence, cell) of every packed token."""
    out = []
    for a, n in enumerate(kv_lengths):
        ql = int(query_starts[a + 1] - query_starts[a])
        out += [(a, int(n) - ql + t) for t in range(ql)]
    return out


def paged_rope(x, positions, axis_of_pair, theta):
    """x [N, H, D] with pair i of every head turned by the angle
    positions[axis_of_pair[i], n] * theta^(-2i/D)."""
    x = np.asarray(x, dtype=np.float64)
    half = x.shape[-1] // 2
    out = np.empty_like(x)
    for i in range(half):
        phi = np.asarray(positions)[axis_of_pair[i]].astype(np.float64) * np.float64(theta) ** (-2.0 * i / (2 * half))
        c, s = np.cos(phi)[:, None], np.sin(phi)[:, None]
        out[..., i] = x[..., i] * c - x[..., i + half] * s
        out[..., i + half] = x[..., i + half] * c + x[..., i] * s
    return out


def _weights(q, k, scale, cells, G):
    """Scores [T, H_q, n] of one sequence, -inf where a token does not see a cell."""
    kk = np.repeat(k, G, axis=0)                                # [H_q, n, D]
    s = np.einsum("thd,hjd->thj", q, kk) * scale
    s[np.broadcast_to(np.arange(k.shape[1])[None, None, :] > np.asarray(cells)[:, None, None], s.shape)] = -np.inf
    return s


def paged_attention(q, k_pool, v_pool, query_starts, kv_lengths, block_table, scale):
    """(out, lse, spread, reach): the attention, the log of its sums, and for
    error bounds sum_j p_j |v_j| and max_j scale * sum_d |q_d k_jd|."""
    N, H_q, D = q.shape
    G = H_q // k_pool.shape[1]
    out, lse = np.full((N, H_q, D), np.nan), np.full((N, H_q), np.nan)
    spread, reach = np.full((N, H_q, D), np.nan), np.full((N, H_q), np.nan)
    for a, n in enumerate(kv_lengths):
        b, e = int(query_starts[a]), int(query_starts[a + 1])
        if e == b:
            continue
        k, v = paged_cells(k_pool, block_table[a], n), paged_cells(v_pool, block_table[a], n)
        s = _weights(q[b:e], k, scale, np.arange(n - (e - b), n), G)
        m = s.max(-1, keepdims=True)
        p = np.exp(s - m)
        l = p.sum(-1, keepdims=True)
        p /= l
        vv = np.repeat(v, G, axis=0)
        out[b:e] = np.einsum("thj,hjd->thd", p, vv)
        spread[b:e] = np.einsum("thj,hjd->thd", p, np.abs(vv))
        lse[b:e] = (m + np.log(l))[..., 0]
        reach[b:e] = np.einsum("thd,hjd->thj", np.abs(q[b:e]), np.abs(np.repeat(k, G, axis=0))).max(-1) * abs(scale)
    return out, lse, spread, reach


def paged_mass(q, lse, k_pool, query_starts, kv_lengths, block_table, scale, M):
    """The weight each cell gets, [A, H_kv, M] (zero where there is none)."""
    G = q.shape[1] // k_pool.shape[1]
    mass = np.zeros((len(kv_lengths), k_pool.shape[1], M))
    for a, n in enumerate(kv_lengths):
        b, e = int(query_starts[a]), int(query_starts[a + 1])
        if e == b:
            continue
        s = _weights(q[b:e], paged_cells(k_pool, block_table[a], n), scale, np.arange(n - (e - b), n), G)
        w = np.exp(s - lse[b:e, :, None])
        mass[a, :, :n] = w.reshape(e - b, -1, G, n).sum((0, 2))
    return mass


def paged_evict(mass, kv_lengths, block_table, keep, recent, k_pool, v_pool):
    """(k_pool', v_pool', mass_out, kept, new_lengths)."""
    A, H_kv, M = mass.shape
    page = k_pool.shape[2]
    k, v = np.array(k_pool), np.array(v_pool)
    mass_out, kept = np.zeros_like(mass), np.full((A, H_kv, keep), -1, dtype=np.int64)
    for a, n in enumerate(int(x) for x in kv_lengths):
        for g in range(H_kv):
            idx = np.arange(n)
            if n > keep:
                old = mass[a, g, :n - recent].astype(np.float64)
                old = np.where(np.isnan(old), -np.inf, old)
                # NaN below even -inf: (is it a number, value) decides, then the cell
                rank = sorted(range(n - recent), key=lambda j: (bool(np.isnan(mass[a, g, j])), -old[j], j))
                idx = np.array(sorted(rank[:keep - recent]) + list(range(n - recent, n)), dtype=np.int64)
                t = np.asarray(block_table[a])
                to = np.arange(keep)
                k[t[to // page], g, to % page] = k_pool[t[idx // page], g, idx % page]
                v[t[to // page], g, to % page] = v_pool[t[idx // page], g, idx % page]
            kept[a, g, :len(idx)] = idx
            mass_out[a, g, :len(idx)] = mass[a, g, idx]
    return k, v, mass_out, kept, np.minimum(np.asarray(kv_lengths), keep)
