"""The operators of the paged key/value cache, as they are measured.

A paged cache keeps the keys and values of many sequences in one pool of pages,
``k_cache``/``v_cache`` [P, H_kv, page, D].  Row a of ``block_table``
[A, max_pages] names sequence a's pages: its cell j is cell ``j % page`` of page
``block_table[a, j // page]``.  The new tokens of all sequences are packed:
sequence a's are rows ``query_starts[a]`` .. ``query_starts[a + 1]`` of q, and
they are the last cells of its ``kv_lengths[a]``.  Four operators work on it:

  store      split-half rotary positions with several axes (pair i of a head
             turns by the position on axis ``axis_of_pair[i]``) for the new
             queries and keys, and the store of keys and values into their cells
  attention  grouped-query attention of a chunk of new tokens (one or many per
             sequence) over the cells up to their own, with the log of the sum
  mass       attention weight that each cell gets from a chunk's queries, added
             to what it has so far
  evict      of each sequence's cells, per KV head, the `recent` last ones and
             those of greatest mass are kept and moved to the front of its pages

`run` computes them in plain torch operations, or calls the library's kernels
where `own` is true; `exact` computes them in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def _case(name, op, dtype, A, hq, hkv, d, page, q, kv, ones=0, mix=1, **more):
    """q, kv: ranges of the sequences' new tokens and of the cells before them;
    `ones` of the A sequences have a single new token."""
    c = {"op": op, "dtype": dtype, "A": A, "hq": hq, "hkv": hkv, "d": d, "page": page, "q_lo": q[0], "q_hi": q[1],
         "kv_lo": kv[0], "kv_hi": kv[1], "ones": ones, "mix": mix}
    c.update(more)
    if name:
        c = {"name": name, **c}
    return c


def listed():
    return [
        # one decode step's store: 32 sequences, one new token each (latency)
        _case("store decode 32", "store", "bf16", 32, 32, 8, 128, 16, (1, 1), (20, 230), theta=500000.0, interleaved=False),
        # chunks of prompts with an image in them, ragged, heads of width 64
        _case("store image chunks", "store", "f16", 5, 16, 4, 64, 32, (301, 1237), (0, 700), theta=10000.0,
              interleaved=True),
        # the store of a prefill of 16 prompts of up to 1024 tokens
        _case("store prefill 16x1024", "store", "bf16", 16, 32, 8, 128, 64, (1021, 1024), (0, 0), theta=500000.0,
              interleaved=False),
        # a decode step of a few short requests (latency)
        _case("decode 4 short", "attention", "f16", 4, 4, 2, 64, 16, (1, 1), (30, 500)),
        # a decode step of 32 requests, contexts up to 4096
        _case("decode 32x4096", "attention", "bf16", 32, 32, 8, 128, 16, (1, 1), (60, 4095)),
        # a decode step over long contexts
        _case("decode 8x65536", "attention", "bf16", 8, 64, 8, 128, 64, (1, 1), (32768, 65535)),
        # one step of continuous batching: chunks of prompts beside decoding requests
        _case("mixed 28", "attention", "bf16", 28, 32, 8, 128, 32, (40, 512), (100, 4000), ones=22),
        # chunks of long prompts over what earlier chunks stored
        _case("chunk 4x2048", "attention", "bf16", 4, 32, 8, 128, 128, (2000, 2048), (6000, 14000)),
        # a decode step's weights, added to the cells' mass
        _case("mass decode 32", "mass", "bf16", 32, 32, 8, 128, 16, (1, 1), (60, 4095)),
        # the weights of a prompt's last tokens, from which its cells are chosen
        _case("mass window 8x64", "mass", "f16", 8, 32, 8, 128, 64, (61, 64), (4000, 16000)),
        # a few requests cut to 256 cells, heads of width 64
        _case("evict 4 to 256", "evict", "f16", 4, 4, 2, 64, 16, (1, 1), (200, 900), keep=256, recent=31),
        # a batch cut to 2048 cells
        _case("evict 32 to 2048", "evict", "bf16", 32, 32, 8, 128, 32, (1, 1), (1500, 8191), keep=2048, recent=128),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    largest = {}
    for c in listed():
        w = work(c)
        x = largest.setdefault(c["op"], [0, 0, 0])
        x[0], x[1], x[2] = max(x[0], w["bytes"]), max(x[1], w["flops"]), max(x[2], _padded(c))
    while True:
        op = rng.choice(["store", "attention", "attention", "mass", "evict"])
        hkv = rng.choice([1, 2, 4, 5, 8])
        g = rng.choice([1, 2, 3, 4, 6, 7, 8, 12, 16])
        kind = {"dtype": rng.choice(["bf16", "f16"]), "A": _spread(rng, 1, 64), "hq": hkv * g, "hkv": hkv,
                "d": rng.choice([64, 128]), "page": rng.choice([16, 32, 64, 128]), "mix": rng.randrange(1 << 20)}
        q_hi = rng.choice([1, _spread(rng, 1, 64), _spread(rng, 1, 2048)])
        kv_hi = _spread(rng, 1, 16000)
        more = {"q": (max(1, q_hi // rng.choice([1, 2, 8])), q_hi), "kv": (kv_hi // rng.choice([1, 2, 10]), kv_hi)}
        if op == "store":
            more |= {"theta": rng.choice([10000.0, 500000.0, 1000000.0]), "interleaved": rng.random() < 0.5,
                     "kv": (0, min(kv_hi, 1000))}
        elif op == "evict":
            keep = _spread(rng, 8, 4096)
            more |= {"q": (1, 1), "keep": keep, "recent": rng.choice([0, rng.randint(0, keep), keep // 16])}
        elif q_hi > 1 and rng.random() < 0.5:
            more["ones"] = kind["A"] // 2
        if op == "mass":
            more["q"] = (min(more["q"][0], 128), min(q_hi, 128))
        c = _case(None, op, **kind, **more)
        w, x = work(c), largest[op]
        if w["bytes"] <= x[0] and w["flops"] <= x[1] and _padded(c) <= x[2]:
            return c


def _lengths(case):
    """Per sequence: new tokens and cells (the new tokens' among them)."""
    r = random.Random("%d %d %d" % (case["mix"], case["A"], case["kv_hi"]))
    ql, kl = [], []
    for a in range(case["A"]):
        q = 1 if a < case["ones"] else _spread(r, case["q_lo"], case["q_hi"])
        ql.append(q)
        kl.append(q + r.randint(case["kv_lo"], case["kv_hi"]))
    order = list(range(case["A"]))
    r.shuffle(order)
    return [ql[i] for i in order], [kl[i] for i in order]


def _max_pages(case):
    return max(-(-n // case["page"]) for n in _lengths(case)[1]) + 1


def _padded(case):
    """Values of the plain form's largest tensor."""
    ql, kl = _lengths(case)
    cells = case["A"] * _max_pages(case) * case["page"] * case["hkv"]
    if case["op"] in ("attention", "mass"):
        return cells * max(case["d"], max(ql) * case["hq"] // case["hkv"])
    return cells * case["d"]


def work(case):
    ql, kl = _lengths(case)
    A, hq, hkv, d, n = case["A"], case["hq"], case["hkv"], case["d"], sum(ql)
    pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(ql, kl))  # (new token, cell that it sees)
    cells = sum(kl)
    table = 4 * (sum(-(-k // case["page"]) for k in kl) + 2 * A + 1)
    if case["op"] == "store":
        return {"bytes": 2 * 2 * n * (hq + 2 * hkv) * d + 4 * 3 * n + table, "flops": 3 * n * (hq + hkv) * d}
    if case["op"] == "attention":
        return {"bytes": 2 * 2 * cells * hkv * d + 2 * 2 * n * hq * d + 4 * n * hq + table, "flops": 4 * pairs * hq * d}
    if case["op"] == "mass":
        return {"bytes": 2 * cells * hkv * d + 2 * n * hq * d + 4 * n * hq + 8 * cells * hkv + table,
                "flops": 2 * pairs * hq * d}
    kept = sum(min(k, case["keep"]) for k in kl)
    moved = sum(case["keep"] for k in kl if k > case["keep"])
    M = _max_pages(case) * case["page"]
    return {"bytes": hkv * (4 * cells + 2 * 2 * 2 * moved * d + 4 * kept + 4 * A * M + 4 * A * case["keep"]) + table,
            "flops": 2 * hkv * cells}


# ------------------------------------------------------------------ inputs
def _axis_of_pair(d, interleaved):
    """Pairs of the three axes (time, height, width): in the ratio 2 : 3 : 3,
    as runs, or by turns until an axis has all its pairs."""
    n = [d // 8, 3 * d // 16, 3 * d // 16]
    if not interleaved:
        return [0] * n[0] + [1] * n[1] + [2] * n[2]
    out, left = [], list(n)
    while len(out) < d // 2:
        for a in range(3):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    dt = DTYPES[case["dtype"]]
    g = torch.Generator(dev).manual_seed(int(seed))
    r = np.random.RandomState(int(seed) % (1 << 32))
    A, hq, hkv, d, page = case["A"], case["hq"], case["hkv"], case["d"], case["page"]
    ql, kl = _lengths(case)
    N, maxp = sum(ql), _max_pages(case)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    # the pages of every sequence, from anywhere in the pool; behind them -1
    need = [-(-n // page) for n in kl]
    P = sum(need) + 3
    ids = r.permutation(P).astype(np.int32)
    table = np.full((A, maxp), -1, np.int32)
    at = 0
    for a in range(A):
        table[a, :need[a]] = ids[at:at + need[a]]
        at += need[a]
    starts = np.concatenate([[0], np.cumsum(ql)]).astype(np.int32)

    def up(x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(dev)

    s = {"case": dict(case), "query_starts": up(starts), "kv_lengths": up(np.array(kl, np.int32)),
         "block_table": up(table), "k_cache": randn(P, hkv, page, d), "v_cache": randn(P, hkv, page, d),
         "max_query_len": max(ql), "scale": 1.0 / math.sqrt(d)}
    # which sequence each new token belongs to, and its cell: host-made index
    # arrays that the plain form and the references use
    seq = np.repeat(np.arange(A), ql)
    cell = np.arange(N) - starts[seq] + (np.array(kl) - np.array(ql))[seq]
    s["seq"], s["cell"] = up(seq.astype(np.int64)), up(cell.astype(np.int64))
    if case["op"] == "store":
        qkv = randn(N, hq + 2 * hkv, d)  # a fused projection's rows: q, k and v are views of them
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        # text, then an image of `width` columns whose patches share a time
        t = np.arange(N) - starts[seq]
        before = (np.array(kl) - np.array(ql))[seq]
        text = np.array([q // 4 for q in ql])[seq]
        width = r.randint(5, 40, A)[seq]
        i = np.maximum(t - text, 0)
        base = before + np.minimum(t, text)
        pos = np.stack([base, base + i // width, base + i % width]).astype(np.int32)
        s["positions"] = up(pos)
        s["axis_of_pair"] = _axis_of_pair(d, case["interleaved"])
    elif case["op"] in ("attention", "mass"):
        s["q_rot"] = randn(N, hq, d)
        if case["op"] == "mass":
            seen = torch.log(s["cell"].float() + 1.0)[:, None]
            s["lse"] = seen + 0.5 + 0.1 * torch.randn(N, hq, generator=g, device=dev)
    if case["op"] in ("mass", "evict"):
        # weight so far: most cells have little of it, some none at all
        M = maxp * page
        m = torch.rand(A, hkv, M, generator=g, device=dev)
        s["mass"] = torch.where(m < 0.1, torch.zeros_like(m), m ** 8 * 4.0)
    if own:  # the caller's output buffers, workspace and prepared call, as a serving loop keeps them
        s["call"], s["outputs"] = _prepare_call(s)
    return s


def _prepare_call(s):
    import kv_cached_gqa_rope_gb300 as kv
    c = s["case"]
    meta = (s["query_starts"], s["kv_lengths"], s["block_table"])
    if c["op"] == "store":
        ws = kv.new_workspace(kv.paged_rope_kv_store_workspace_size())
        q_out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
        return kv.prepare_paged_rope_kv_store_out_(
            s["q"], s["k"], s["v"], s["positions"], *meta, c["theta"], s["axis_of_pair"], q_out, s["k_cache"],
            s["v_cache"], ws), (q_out, s["k_cache"], s["v_cache"])
    if c["op"] == "attention":
        ws = kv.new_workspace(kv.paged_gqa_attention_workspace_size(c["hq"], c["hkv"], c["d"]))
        out = torch.empty_like(s["q_rot"])
        lse = torch.empty(out.shape[:2], dtype=torch.float32, device="cuda")
        return kv.prepare_paged_gqa_attention_out_(
            s["q_rot"], s["k_cache"], s["v_cache"], *meta, s["max_query_len"], s["scale"], out, lse, ws), (out, lse)
    if c["op"] == "mass":
        ws = kv.new_workspace(kv.paged_attention_mass_workspace_size())
        return kv.prepare_paged_attention_mass_out_(
            s["q_rot"], s["lse"], s["k_cache"], *meta, s["max_query_len"], s["scale"], s["mass"], ws), (s["mass"],)
    ws = kv.new_workspace(kv.paged_evict_workspace_size(c["A"], c["hkv"], c["keep"]))
    mass_out = torch.empty_like(s["mass"])
    kept = torch.empty(c["A"], c["hkv"], c["keep"], dtype=torch.int32, device="cuda")
    lengths = torch.empty(c["A"], dtype=torch.int32, device="cuda")
    return kv.prepare_paged_evict_out_(
        s["mass"], s["kv_lengths"], s["block_table"], c["keep"], c["recent"], s["k_cache"], s["v_cache"], mass_out,
        kept, lengths, ws), (s["k_cache"], s["v_cache"], mass_out, kept, lengths)


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        state["call"]()
        return state["outputs"]
    return {"store": _store, "attention": _attention, "mass": _mass, "evict": _evict}[state["case"]["op"]](state)


def _turn(x, cos, sin):
    h = x.shape[-1] // 2
    a, b = x[..., :h].float(), x[..., h:].float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(x.dtype)


def _store(s):
    c = s["case"]
    half = c["d"] // 2
    axis = torch.tensor(s["axis_of_pair"], device="cuda")
    freq = c["theta"] ** (-2.0 * torch.arange(half, device="cuda", dtype=torch.float64) / c["d"])
    angle = s["positions"].double()[axis].T * freq  # [N, half]; 32 bits lose far positions' angles
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q_out = _turn(s["q"], cos, sin)
    pid = s["block_table"][s["seq"], s["cell"] // c["page"]].long()
    off = s["cell"] % c["page"]
    s["k_cache"][pid, :, off] = _turn(s["k"], cos, sin)
    s["v_cache"][pid, :, off] = s["v"]
    return q_out, s["k_cache"], s["v_cache"]


def _dense(s, cache):
    """The cells of every sequence side by side, [A, H_kv, max_pages * page, D]
    in 32 bits; cells behind a sequence's length read as zeros."""
    x = cache[s["block_table"].clamp(min=0).long()]  # [A, max_pages, H_kv, page, D]
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)
    live = torch.arange(x.shape[2], device="cuda") < s["kv_lengths"][:, None]
    return torch.where(live[:, None, :, None], x, torch.zeros((), dtype=x.dtype, device="cuda")).float()


def _scores(s):
    """Scaled scores of the padded queries, [A, H_kv, T * G, cells], minus
    infinity where a query does not see a cell, and each token's place."""
    c = s["case"]
    A, hkv, G, T = c["A"], c["hkv"], c["hq"] // c["hkv"], s["max_query_len"]
    t = torch.arange(s["seq"].numel(), device="cuda") - s["query_starts"].long()[s["seq"]]
    q = torch.zeros(A, T, hkv, G, c["d"], device="cuda")
    q[s["seq"], t] = s["q_rot"].float().unflatten(1, (hkv, G))
    sc = q.permute(0, 2, 1, 3, 4).flatten(2, 3) @ _dense(s, s["k_cache"]).transpose(2, 3)
    sc *= s["scale"]
    last = torch.full((A, T), -1, device="cuda", dtype=torch.int64)
    last[s["seq"], t] = s["cell"]
    hidden = torch.arange(sc.shape[3], device="cuda") > last[:, :, None]
    sc.unflatten(2, (T, G)).masked_fill_(hidden[:, None, :, None], float("-inf"))
    return sc, t


def _attention(s):
    c = s["case"]
    hkv, G, T = c["hkv"], c["hq"] // c["hkv"], s["max_query_len"]
    sc, t = _scores(s)
    m = sc.amax(-1, keepdim=True).clamp(min=-3e38)  # a padded query sees nothing
    sc -= m
    p = sc.exp_()
    l = p.sum(-1, keepdim=True)
    o = (p @ _dense(s, s["v_cache"])) / l
    o = o.unflatten(2, (T, G)).permute(0, 2, 1, 3, 4)[s["seq"], t].flatten(1, 2)
    lse = (m + l.log()).squeeze(-1).unflatten(2, (T, G)).permute(0, 2, 1, 3)[s["seq"], t].flatten(1, 2)
    return o.to(DTYPES[c["dtype"]]), lse


def _mass(s):
    c = s["case"]
    hkv, G, T = c["hkv"], c["hq"] // c["hkv"], s["max_query_len"]
    sc, t = _scores(s)
    lse = torch.zeros(c["A"], T, hkv, G, device="cuda")
    lse[s["seq"], t] = s["lse"].unflatten(1, (hkv, G))
    sc -= lse.permute(0, 2, 1, 3).flatten(2, 3).unsqueeze(-1)
    s["mass"] += sc.exp_().sum(2)
    return (s["mass"],)


def _evict(s):
    c = s["case"]
    keep, recent, page = c["keep"], c["recent"], c["page"]
    n = s["kv_lengths"].long()[:, None, None]
    M = s["mass"].shape[2]
    j = torch.arange(M, device="cuda")
    # recent cells first of all, cells behind the length last; a stable sort leaves ties to the lowest cell
    rank = torch.where(j >= n - recent, float("inf"), s["mass"])
    rank = torch.where(j >= n, float("-inf"), rank)
    first = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :min(keep, M)]
    first = torch.where(first < n, first, M).sort(-1).values  # the kept cells in their order, M where there are fewer
    pad = torch.full((*first.shape[:2], keep - first.shape[2]), M, device="cuda")
    first = torch.cat([first, pad], -1)
    some = first < M
    kept = torch.where(some, first, -1)
    src = first.clamp(max=M - 1)
    mass_out = torch.zeros_like(s["mass"])
    w = min(keep, M)
    mass_out[..., :w] = torch.where(some, torch.gather(s["mass"], 2, src), 0.0)[..., :w]
    a, h, i = torch.nonzero(some & (n > keep), as_tuple=True)
    frm, table = src[a, h, i], s["block_table"].long()
    pf, pt = table[a, frm // page], table[a, i // page]
    for x in (s["k_cache"], s["v_cache"]):
        x[pt, h, i % page] = x[pf, h, frm % page]
    return s["k_cache"], s["v_cache"], mass_out, kept.int(), s["kv_lengths"].clamp(max=keep)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"store": _exact_store, "attention": _exact_attention, "mass": _exact_mass,
            "evict": _exact_evict}[case["op"]](s)


def _cells(s, a, cache):
    """Sequence a's cells in order, [H_kv, n, D] in 64 bits."""
    n, page = int(s["kv_lengths"][a]), s["case"]["page"]
    ids = s["block_table"][a, :-(-n // page)].long()
    x = torch.cat([cache[i] for i in ids], 1)
    return x[:, :n].double()


def _exact_store(s):
    c = s["case"]
    half = c["d"] // 2
    N = s["q"].shape[0]
    unit = torch.zeros(N, half, dtype=torch.complex128, device="cuda")
    for i in range(half):
        f = math.exp(-2.0 * i / c["d"] * math.log(c["theta"]))
        x = s["positions"][s["axis_of_pair"][i]].double() * f
        unit[:, i] = torch.polar(torch.ones_like(x), x)

    def turned(x):
        z = torch.complex(x[..., :half].double(), x[..., half:].double()) * unit[:, None]
        return torch.cat([z.real, z.imag], -1)

    k, v = s["k_cache"].double(), s["v_cache"].double()
    kn, cell, seq, table = turned(s["k"]), s["cell"].tolist(), s["seq"].tolist(), s["block_table"].tolist()
    at = torch.tensor([[table[a][j // c["page"]], j % c["page"]] for a, j in zip(seq, cell)], device="cuda")
    k.transpose(1, 2)[at[:, 0], at[:, 1]] = kn
    v.transpose(1, 2)[at[:, 0], at[:, 1]] = s["v"].double()
    return turned(s["q"]), k, v


def _exact_rows(s, a, g):
    """Scores of sequence a's queries that read KV head g, [rows, G, cells] in
    64 bits, a few hundred queries at a time, with the queries' places."""
    G = s["case"]["hq"] // s["case"]["hkv"]
    q0, q1, n = int(s["query_starts"][a]), int(s["query_starts"][a + 1]), int(s["kv_lengths"][a])
    k = _cells(s, a, s["k_cache"])[g]
    for b in range(q0, q1, 512):
        e = min(q1, b + 512)
        x = torch.einsum("tgd,jd->tgj", s["q_rot"][b:e, g * G:(g + 1) * G].double(), k) * s["scale"]
        sees = torch.arange(n, device="cuda") <= (n - q1 + torch.arange(b, e, device="cuda"))[:, None]
        yield b, e, torch.where(sees[:, None], x, float("-inf"))


def _exact_attention(s):
    c = s["case"]
    G = c["hq"] // c["hkv"]
    if work(c)["flops"] > 6e12:
        return None
    out = torch.zeros(s["q_rot"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device="cuda")
    for a in range(c["A"]):
        v = _cells(s, a, s["v_cache"])
        for g in range(c["hkv"]):
            for b, e, x in _exact_rows(s, a, g):
                y = torch.logsumexp(x, -1)
                out[b:e, g * G:(g + 1) * G] = torch.einsum("tgj,jd->tgd", (x - y[..., None]).exp(), v[g])
                lse[b:e, g * G:(g + 1) * G] = y
    return out, lse


def _exact_mass(s):
    c = s["case"]
    G = c["hq"] // c["hkv"]
    mass = s["mass"].double()
    for a in range(c["A"]):
        n = int(s["kv_lengths"][a])
        for g in range(c["hkv"]):
            for b, e, x in _exact_rows(s, a, g):
                mass[a, g, :n] += (x - s["lse"][b:e, g * G:(g + 1) * G, None].double()).exp().sum((0, 1))
    return (mass,)


def _exact_evict(s):
    c = s["case"]
    keep, recent, page = c["keep"], c["recent"], c["page"]
    k0, v0 = s["k_cache"], s["v_cache"]
    k, v = k0.double(), v0.double()
    mass, table = s["mass"].cpu().numpy().astype(np.float64), s["block_table"].cpu().numpy()
    mass_out = np.zeros_like(mass)
    kept = np.full((c["A"], c["hkv"], keep), -1, np.int64)
    lens = s["kv_lengths"].cpu().numpy()
    for a, n in enumerate(lens):
        for g in range(c["hkv"]):
            m = mass[a, g, :n]
            if n > keep:
                old = n - recent
                order = np.lexsort((np.arange(old), -m[:old]))[:keep - recent]
                idx = np.sort(np.concatenate([order, np.arange(old, n)]))
                src = torch.from_numpy(np.stack([table[a][idx // page], idx % page])).cuda().long()
                to = np.arange(keep)
                dst = torch.from_numpy(np.stack([table[a][to // page], to % page])).cuda().long()
                k[dst[0], g, dst[1]] = k0[src[0], g, src[1]].double()
                v[dst[0], g, dst[1]] = v0[src[0], g, src[1]].double()
            else:
                idx = np.arange(n)
            kept[a, g, :len(idx)] = idx
            mass_out[a, g, :len(idx)] = m[idx]
    return (k, v, torch.from_numpy(mass_out), torch.from_numpy(kept), torch.from_numpy(np.minimum(lens, keep)))
