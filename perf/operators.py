"""Cases of the paged decode cache's operators: what a serving program does at every
token with keys and values held in pages of S tokens, a page table a sequence and
reference counts, all on the device.

Kinds of case (``case["op"]``):

* ``attn``: attention of one new token a sequence over its whole cache (a dense
  layer, a sequence too short to select from, or the exact answer beside the sparse
  step); ``append`` true writes the token's key and value rows on the way.
* ``step``: the pyramid step over pages (append, summaries, selection, attention).
  Keys carry planted leaves, as in the repository's retrieval workload, so that the
  kept leaves are the forced and the planted ones by a wide margin.
* ``append``: rows of new tokens into the pages of every sequence.
* ``fork``: a beam step: the survivors' rows are shared with their children, every
  sequence gets room for one more token (a shared last page is copied).
* ``admit``: finished sequences leave, new prompts get pages and their rows.
* ``compact``: live pages move to the low end of the pool.

Page tables are scattered (pages in random order), as they are after some time of
service. The calls that change table and counts first put back the integers that
``prepare`` made, so that every pass does the same work.
"""
import math

import numpy as np
import torch

own = False

#: words kept free at the head of a list of moves: count, pages missing, pages live, pages free
HEAD = 4


# ---- cases ----------------------------------------------------------------------------

def _case(name, op, **kw):
    base = {"op": op, "B": 1, "Hq": 8, "Hkv": 8, "d": 128, "S": 64, "N": 16384, "dtype": "bf16", "lens": "full",
            "C": 64, "K": 16, "append": False, "T": 1, "fill": 0.5}
    base.update(kw)
    return dict(base, name=name) if name else base


def listed():
    return [
        # one short chat turn: what counts is latency
        _case("attn_one_short", "attn", B=1, N=1024, lens="full"),
        # one sequence of the longest context: the split over its length has to fill the GPU
        _case("attn_one_256k", "attn", B=1, N=262144),
        # a serving batch of very unequal lengths, an empty slot and a one-token sequence among them
        _case("attn_ragged_gqa32x8", "attn", B=64, Hq=32, Hkv=8, S=16, lens="ragged"),
        # fp32, narrow heads, a page size that no tile divides, token appended on the way
        _case("attn_append_f32", "attn", B=16, Hq=8, Hkv=2, d=64, S=48, N=4000, dtype="f32", lens="ragged", append=True),
        # a full batch of long sequences
        _case("attn_64x16k_gqa32x8", "attn", B=64, Hq=32, Hkv=8),
        # the sparse step of a full batch (the repository's MHA-8 heads)
        _case("step_64x16k_mha8", "step", B=64, lens="near"),
        # the sparse step of a few small sequences in fp32
        _case("step_small_f32", "step", B=3, Hq=4, Hkv=2, d=64, C=16, K=4, S=32, N=1024, dtype="f32", lens="near"),
        # one token's rows for a full batch: latency
        _case("append_token", "append", B=64, N=2048, lens="near"),
        # prompts of a small batch out of a prefill
        _case("append_prompt", "append", B=4, S=16, T=8192, lens="full"),
        # a beam step of 64 rows
        _case("fork_beam", "fork", B=64, N=4096, lens="near"),
        # half of the slots get new prompts
        _case("admit_prompts", "admit", B=32, T=2048, N=8192, lens="ragged"),
        # defragmenting a half-empty pool
        _case("compact_pool", "compact", B=32, N=8192, lens="near", fill=0.5),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "step", "append", "fork", "admit", "compact"])
    G = rng.choice([1, 2, 4, 8, 16])
    c = {"Hkv": rng.choice([1, 2, 4, 8]), "d": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "bf16", "f32"]),
         "lens": rng.choice(["full", "near", "ragged"])}
    c["Hq"] = c["Hkv"] * G
    c["B"] = _spread(rng, 1, 64)
    # at most 2^22 cached rows of all heads together
    c["N"] = max(16, _spread(rng, 16, max(32, min(262144, (1 << 22) // (c["B"] * c["Hkv"])))))
    c["S"] = rng.choice([8, 16, 32, 64, 128, rng.randrange(1, 100)])
    if op == "attn":
        c["append"] = c["B"] * c["N"] * c["Hkv"] <= (1 << 20) and rng.random() < 0.5
    if op == "step":
        c["C"] = rng.choice([16, 32, 64])
        c["K"] = rng.choice([4, 8, 16])
        c["S"] = c["C"] * rng.choice([1, 2])
        c["N"] = min(max(c["N"], 4 * c["C"]), 32768)
        c["lens"] = "near"
    if op in ("append", "admit"):
        c["T"] = _spread(rng, 1, max(2, c["N"] // 2))
    if op in ("fork", "admit", "compact"):
        c["N"] = min(c["N"], 16384)
        c["T"] = min(c.get("T", 1), c["N"] // 2)
        c["S"] = max(c["S"], 8)
        c["fill"] = rng.choice([0.25, 0.5, 0.9])
    return _case(None, op, **c)


def _lens(case):
    """Cached tokens of each sequence, the token in hand included: a rule of the case alone."""
    B, N, kind = case["B"], case["N"], case["lens"]
    b = np.arange(B)
    frac = np.modf((b + 1) * 0.6180339887)[0]
    if kind == "full":
        n = N - (b * 7) % max(1, N // 50)
    elif kind == "near":
        n = N - np.floor(frac * (N // 4)).astype(np.int64)
    else:
        n = np.round(N ** frac).astype(np.int64)
        if B >= 8 and case["op"] in ("attn", "append"):
            n[1], n[2] = 0, 1
    n = np.clip(n, 0, N)
    if case["op"] in ("fork", "admit"):  # room for what is added
        n = np.clip(n, 1, N - max(1, case["T"] if case["op"] == "admit" else 1))
    return n.astype(np.int64)


def _counts(case):
    """Rows appended to each sequence (append) or wanted by each new prompt (admit)."""
    n, T = _lens(case), case["T"]
    b = np.arange(case["B"])
    if case["op"] == "append":
        return np.minimum(n, T) if T > 1 else np.minimum(n, 1)
    want = np.maximum(1, T - (b * 37) % max(1, T // 2))
    return np.where(b % 2 == 0, np.minimum(want, case["N"]), 0)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _width(case):
    return -(-case["N"] // case["S"])


def _levels(N, C):
    M, off = [-(-N // C)], [0]
    while M[-1] > 1:
        off.append(off[-1] + M[-1])
        M.append(-(-M[-1] // 2))
    return M, off


def work(case):
    """Bytes read once and written once, and products, that one pass cannot do without."""
    es = 2 if case["dtype"] == "bf16" else 4
    n, S, d, Hq, Hkv, B = _lens(case), case["S"], case["d"], case["Hq"], case["Hkv"], case["B"]
    row = Hkv * d * es * 2  # a token's key and value rows
    pages = int(np.sum(-(-n // S)))
    op = case["op"]
    if op == "attn":
        fl = 4.0 * float(n.sum()) * Hq * d
        b = float(n.sum()) * row + 2 * B * Hq * d * es + 4 * B * Hq + 4 * pages + (B * row if case["append"] else 0)
        return {"bytes": b, "flops": fl}
    if op == "step":  # scored summaries, the raw keys of level-1 candidates, values of the kept leaves
        C, K = case["C"], case["K"]
        M, _ = _levels(case["N"], C)
        b = fl = 0.0
        for x in n:
            scored = sum(1 for m in range(1, len(M)) if -(-int(x) // (C << m)) > K)
            leaves = min(2 * K, -(-int(x) // C))
            kept = min(K, leaves)
            b += Hkv * (scored * 2 * K * 2 * d * 4 + leaves * C * d * es + kept * C * d * es + len(M) * d * 4) + 2 * row
            fl += Hq * d * (scored * 4 * K * 2 + 2 * leaves * C + 2 * kept * C)
        return {"bytes": b + 2 * B * Hq * d * es + 4 * B * Hkv * K, "flops": fl}
    if op == "append":
        return {"bytes": 2.0 * float(_counts(case).sum()) * row + 4 * B * 2, "flops": 0}
    table = 4.0 * B * _width(case)
    if op == "fork":  # old and new table; about half of the rows copy a page
        return {"bytes": 2 * table + B / 2 * S * row * 2, "flops": 0}
    if op == "admit":
        return {"bytes": table + 2.0 * float(_counts(case).sum()) * row, "flops": 0}
    moved = pages * (1 - case["fill"])  # a live page lies past the live count with that chance
    return {"bytes": 2 * table + 2 * moved * S * row, "flops": 0}


# ---- what a program has in hand ----------------------------------------------------------

def _state_words(P):
    """Words of the page state: counts, the bitmap of free pages, room the library works in."""
    p4, b4 = -(-P // 4) * 4, -(-(-(-P // 32)) // 4) * 4
    return p4, b4, 2 * p4 + 3 * b4 + 16


def _tables(case, seed):
    """Table [B, W], pool size, counts a page: pages in random order, shared where the case shares them."""
    rng = np.random.default_rng(seed)
    B, S, W, op = case["B"], case["S"], _width(case), case["op"]
    n = _lens(case)
    have = -(-n // S)
    table = np.full((B, W), -1, np.int64)
    if op == "fork":  # groups of four rows share the first half of the shortest one's pages
        rank = 0
        for g in range(0, B, 4):
            rows = range(g, min(B, g + 4))
            common = int(min(n[r] for r in rows)) // S // 2
            table[list(rows), :common] = np.arange(rank, rank + common)
            rank += common
            for r in rows:
                table[r, common:have[r]] = np.arange(rank, rank + have[r] - common)
                rank += int(have[r] - common)
        used = rank
    else:
        flat = np.arange(W)[None, :] < have[:, None]
        used = int(flat.sum())
        table[flat] = np.arange(used)
    spare = {"fork": 2 * B + 8, "admit": B * (-(-case["T"] // S) + 1) + 8}.get(op, 5)
    P = used + spare if op != "compact" else max(used + 1, int(used / case["fill"]))
    place = rng.permutation(P)
    table = np.where(table >= 0, place[np.clip(table, 0, None)], -1)
    refs = np.bincount(table[table >= 0], minlength=P).astype(np.int64)
    return table, refs, P


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, Hq, Hkv, d, S, N, op = (case[k] for k in ("B", "Hq", "Hkv", "d", "S", "N", "op"))
    dt, W = _dtype(case), _width(case)
    table, refs, P = _tables(case, seed)
    p4, b4, words = _state_words(P)
    # the integers of the cache, one after another: page state, table, lengths
    ints = np.zeros(words + -(-B * W // 4) * 4 + -(-B // 4) * 4, np.int32)
    ints[:P] = refs
    free = np.zeros(b4 * 32, bool)
    free[:P] = refs == 0
    ints[p4:p4 + b4] = (free.reshape(-1, 32) * (np.uint64(1) << np.arange(32, dtype=np.uint64))).sum(1).astype(np.uint32).view(np.int32)
    at = words + -(-B * W // 4) * 4
    ints[words:words + B * W] = table.reshape(-1)
    ints[at:at + B] = _lens(case)
    ints0 = torch.from_numpy(ints).to(dev)
    ints = ints0.clone()
    s = {"case": case, "P": P, "ints0": ints0, "ints": ints, "state": ints[:words],
         "table": ints[words:words + B * W].view(B, W), "lens": ints[at:at + B]}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=dt)

    s["K"], s["V"] = randn(P, Hkv, S, d), randn(P, Hkv, S, d)
    if op in ("attn", "step"):
        s["q"] = randn(B, Hq, d)
        s["k_new"], s["v_new"] = randn(B, Hkv, d), randn(B, Hkv, d)
        s["o"] = torch.empty(B, Hq, d, device=dev, dtype=dt)
        s["lse"] = torch.empty(B, Hq, device=dev)
    if op == "step":
        _plant(s, g)
    if op in ("append", "admit"):
        s["count"] = torch.from_numpy(_counts(case)).to(dev, torch.int32)
        s["k_new"], s["v_new"] = randn(B, Hkv, case["T"], d), randn(B, Hkv, case["T"], d)
    if op in ("fork", "admit"):
        s["grant"] = torch.empty(B, dtype=torch.int32, device=dev)
    if op in ("fork", "admit", "compact"):
        s["most"] = P // 2 if op == "compact" else B
        s["moves"] = torch.zeros(HEAD + 2 * s["most"], dtype=torch.int32, device=dev)
    if op == "fork":  # the survivors of each group of four rows
        r = np.random.default_rng(seed + 1)
        b = np.arange(B)
        s["parent"] = torch.from_numpy(np.minimum(b // 4 * 4 + r.integers(0, 4, B), B - 1)).to(dev, torch.int32)
        s["add"] = torch.ones(B, dtype=torch.int32, device=dev)
        s["table_out"], s["lens_out"] = torch.empty_like(s["table"]), torch.empty_like(s["lens"])
    if op == "admit":
        s["leave"] = torch.arange(0, B, 2, dtype=torch.int32, device=dev)
    if own:
        from hierarchical_block_sparse_b200 import pisa
        s["cfg"] = pisa.make_cfg(B=B, Hq=Hq, Hkv=Hkv, N=N, d=d, C=case["C"], K=case["K"], dtype=dt)
        s["pages"] = pisa.make_pages(S, P)
        if op == "attn":
            s["ws"] = pisa.alloc_paged_workspace(s["cfg"], s["pages"], dev)
    return s


def _plant(s, g):
    """Queries along a direction of their own, K - 3 leaves a head whose keys follow it, and the summaries of what is cached before the new token."""
    case, K, table, lens = s["case"], s["K"], s["table"].long(), s["lens"].long()
    B, Hq, Hkv, d, S, C = (case[k] for k in ("B", "Hq", "Hkv", "d", "S", "C"))
    dev = K.device
    u = torch.randn(B, Hkv, d, generator=g, device=dev)
    u = u / u.norm(dim=-1, keepdim=True)
    owner = torch.zeros(s["P"], dtype=torch.long, device=dev)
    rows = torch.arange(B, device=dev)[:, None].expand_as(table)
    owner[table[table >= 0]] = rows[table >= 0]
    U = u[owner][:, :, None, :]
    x = K.float()
    x = x - (x * U).sum(-1, keepdim=True) * U
    M1 = _levels(case["N"], C)[0][0]
    cur = (lens - 1) // C
    leaf = torch.arange(M1, device=dev)
    open_ = (leaf[None, :] >= 1) & (leaf[None, :] <= cur[:, None] - 2)
    chance = torch.rand(B, Hkv, M1, generator=g, device=dev) + (~open_)[:, None, :] * 2.0
    n = min(case["K"] - 3, M1)
    pick = chance.topk(n, largest=False)
    tok = (pick.indices[..., None] * C + torch.arange(C, device=dev)).clamp(max=case["N"] - 1)
    live = (pick.values < 1.5)[..., None].expand_as(tok)
    page = table[torch.arange(B, device=dev)[:, None, None, None], tok // S]
    h = torch.arange(Hkv, device=dev)[None, :, None, None].expand_as(tok)
    up = (12.0 * u)[:, :, None, None, :].expand(*tok.shape, d)
    x.index_put_((page[live], h[live], (tok % S)[live]), up[live], accumulate=True)
    K.copy_(x)
    q = 8.0 * u[:, :, None, :] + 0.25 * torch.randn(B, Hkv, Hq // Hkv, d, generator=g, device=dev)
    s["q"].copy_(q.reshape(B, Hq, d))
    k = s["k_new"].float()
    s["k_new"].copy_(k - (k * u).sum(-1, keepdim=True) * u)
    del x
    s["idx"] = torch.empty(B, Hkv, case["K"], dtype=torch.int32, device=dev)
    s["pyr"] = _pyramid(K, table, lens - 1, case, torch.float32).float()


def _pyramid(K, table, lens, case, dt):
    """Summaries of the first lens[b] tokens, laid out for N tokens; zeros where there are none."""
    M, off = _levels(case["N"], case["C"])
    C, B, Hkv, d = case["C"], case["B"], case["Hkv"], case["d"]
    out = torch.zeros(B, Hkv, off[-1] + M[-1], d, device=K.device, dtype=dt)
    for b in range(B):
        n = int(lens[b])
        x = K[table[b].clamp(min=0)].transpose(0, 1).reshape(Hkv, -1, d)[:, :n].to(dt)
        m = -(-n // C)
        x = torch.nn.functional.pad(x, (0, 0, 0, m * C - n)).view(Hkv, m, C, d).sum(2)
        size = (n - torch.arange(m, device=K.device, dtype=dt) * C).clamp(max=C)
        x = x / size[:, None]
        for lv in range(len(M)):
            out[b, :, off[lv]:off[lv] + x.shape[1]] = x
            odd = x[:, -1:] if x.shape[1] % 2 else x[:, :0]
            x = torch.cat([(x[:, 0:x.shape[1] - 1:2] + x[:, 1::2]) * 0.5, odd], 1) if x.shape[1] > 1 else x
    return out


# ---- the plain forms -----------------------------------------------------------------------

def _put_rows(pool, rows, table, lens, count):
    """Writes rows[b, :, i] at token lens[b] - count[b] + i, i < count[b]."""
    B, Hkv, T, _ = rows.shape
    S = pool.shape[2]
    i = torch.arange(T, device=pool.device)
    tok = (lens - count)[:, None] + i
    live = i < count[:, None]
    page = table.gather(1, (tok // S).clamp(0, table.shape[1] - 1))
    at = live.nonzero(as_tuple=True)
    pool[page[at], :, (tok % S)[at]] = rows.transpose(1, 2)[at]


def _get_rows(pool, table, tok):
    """Rows of the tokens tok [B, Hkv, n] in 32 bits."""
    B, Hkv, n = tok.shape
    S = pool.shape[2]
    page = table[:, None, :].expand(B, Hkv, table.shape[1]).gather(2, tok // S).clamp(min=0)
    return pool[page, torch.arange(Hkv, device=pool.device)[None, :, None], tok % S].float()


def _plain_attn(s):
    case, table, lens = s["case"], s["table"].long(), s["lens"].long()
    B, Hq, Hkv, d = (case[k] for k in ("B", "Hq", "Hkv", "d"))
    if case["append"]:
        one = (lens > 0).long()
        _put_rows(s["K"], s["k_new"][:, :, None], table, lens, one)
        _put_rows(s["V"], s["v_new"][:, :, None], table, lens, one)

    def rows(pool):
        return pool[table.clamp(min=0)].transpose(1, 2).reshape(B, Hkv, -1, d).float()

    q = s["q"].float().view(B, Hkv, Hq // Hkv, d)
    z = (q @ rows(s["K"]).transpose(2, 3)) / math.sqrt(d)
    seen = torch.arange(z.shape[-1], device=z.device) < lens[:, None]
    z = z.masked_fill(~seen[:, None, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m.masked_fill(m == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    o = (p @ rows(s["V"])) / total.clamp(min=1e-30)
    lse = (m + torch.log(total)).view(B, Hq)
    o = o.view(B, Hq, d).to(s["o"].dtype)
    return {"o": o, "lse": lse, "K": s["K"], "V": s["V"]} if case["append"] else {"o": o, "lse": lse}


def _plain_step(s):
    case, table, lens = s["case"], s["table"].long(), s["lens"].long()
    B, Hq, Hkv, d, C, K = (case[k] for k in ("B", "Hq", "Hkv", "d", "C", "K"))
    G, dev, pyr = Hq // Hkv, table.device, s["pyr"]
    M, off = _levels(case["N"], C)
    one = torch.ones_like(lens)
    _put_rows(s["K"], s["k_new"][:, :, None], table, lens, one)
    _put_rows(s["V"], s["v_new"][:, :, None], table, lens, one)
    n, cur, b = lens, (lens - 1) // C, torch.arange(B, device=dev)
    # the new token's leaf, then its ancestors: means of what exists
    inside = torch.arange(C, device=dev)
    tok = (cur[:, None] * C + inside)
    live = tok < n[:, None]
    x = _get_rows(s["K"], table, tok.clamp(max=case["N"] - 1)[:, None].expand(B, Hkv, C))
    x = x.masked_fill(~live[:, None, :, None], 0.0).sum(2) / live.sum(1)[:, None, None]
    pyr[b, :, cur] = x
    for lv in range(1, len(M)):
        node = cur >> lv
        left, right = pyr[b, :, off[lv - 1] + 2 * node], pyr[b, :, off[lv - 1] + (2 * node + 1).clamp(max=M[lv - 1] - 1)]
        both = ((2 * node + 1) * (C << (lv - 1)) < n)[:, None, None]
        pyr[b, :, off[lv] + node] = torch.where(both, (left + right) * 0.5, left)
    # the walk: K kept of at most 2K candidates at every level
    q = s["q"].float().view(B, Hkv, G, d) / math.sqrt(d)
    cand = torch.full((B, Hkv, 2 * K), -1, dtype=torch.long, device=dev)
    cand[:, :, 0] = 0
    hh = torch.arange(Hkv, device=dev)[None, :, None]
    for lv in range(len(M) - 1, -1, -1):
        nn = n[:, None, None]
        valid = (cand >= 0) & (cand * (C << lv) < nn)
        c = cand.clamp(min=0)
        if lv > 0:
            child = (2 * c[..., None] + torch.arange(2, device=dev)).view(B, Hkv, -1)
            there = child * (C << (lv - 1)) < nn
            row = pyr[b[:, None, None], hh, off[lv - 1] + child.clamp(max=M[lv - 1] - 1)]
            per = 2
        else:
            child = (c[..., None] * C + inside).view(B, Hkv, -1)
            there = child < nn
            row = _get_rows(s["K"], table, child.clamp(max=case["N"] - 1))
            per = C
        z = (q @ row.transpose(2, 3)).masked_fill(~there[:, :, None], -math.inf)
        score = torch.logsumexp(z.view(B, Hkv, G, 2 * K, per), -1).sum(2)
        forced = (c == 0) | (c == (cur >> lv)[:, None, None]) | ((cur >= 1)[:, None, None] & (c == ((cur - 1).clamp(min=0) >> lv)[:, None, None]))
        score = score.masked_fill(forced, math.inf).masked_fill(~valid, -math.inf)
        order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :K]
        kept = cand.gather(2, order).masked_fill(~valid.gather(2, order), 1 << 40).sort(-1).values
        gone = kept == 1 << 40
        cand = (2 * kept[..., None] + torch.arange(2, device=dev)).masked_fill(gone[..., None], -1).view(B, Hkv, 2 * K)
    kept = kept.masked_fill(gone, -1)
    tok = (kept.clamp(min=0)[..., None] * C + inside)
    seen = ((kept >= 0)[..., None] & (tok < n[:, None, None, None])).view(B, Hkv, 1, K * C)
    tok = tok.view(B, Hkv, K * C).clamp(max=case["N"] - 1)
    z = (q @ _get_rows(s["K"], table, tok).transpose(2, 3)).masked_fill(~seen, -math.inf)
    o = torch.softmax(z, -1) @ _get_rows(s["V"], table, tok)
    return {"idx": kept.int(), "o": o.view(B, Hq, d).to(s["o"].dtype), "pyr": pyr}


def _plain_reserve(refs, table, lens, add, S, N, most):
    """Room for add[b] more tokens a sequence, in order of b: lowest free pages first, a shared last page replaced by a copy."""
    B, W = table.shape
    dev = table.device
    ok = (add > 0) & (lens + add <= N)
    add = add * ok
    have, want = (lens + S - 1) // S, (lens + add + S - 1) // S
    tail = table.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    part = ok & (lens % S != 0)
    same = (tail[:, None] == tail[None, :]) & part[:, None] & part[None, :]
    before = torch.tril(same, -1).sum(1)
    copy = part & (before < refs[tail.clamp(min=0)] - 1)
    need = (want - have) * ok + copy
    base = need.cumsum(0) - need
    free = torch.sort((refs != 0).int(), stable=True).indices
    spare = (refs == 0).sum()
    fits = need.sum() <= spare
    col = torch.arange(W, device=dev)
    at_tail = copy[:, None] & (col == have[:, None] - 1)
    new = (at_tail | ((col >= have[:, None]) & (col < want[:, None]))) & fits
    k = base[:, None] + torch.where(at_tail, 0, copy[:, None] + col - have[:, None])
    page = free[k.clamp(0, free.numel() - 1)]
    out = torch.where(new, page, table)
    copy, grant = copy & fits, add * fits
    refs = refs.scatter_add(0, page.reshape(-1), new.reshape(-1).long()).scatter_add(0, tail.clamp(min=0), -copy.long())
    moves = torch.zeros(HEAD + 2 * most + 2, dtype=torch.long, device=dev)
    slot = torch.where(copy, HEAD + 2 * (copy.cumsum(0) - 1), HEAD + 2 * most)
    moves[slot], moves[slot + 1] = tail, page.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    live = (refs > 0).sum()
    moves[:HEAD] = torch.stack([copy.sum(), (need.sum() - spare).clamp(min=0), live, refs.numel() - live])
    return refs, out, lens + grant, grant, moves[:HEAD + 2 * most].int()


def _plain_copy(s, moves):
    n = int(moves[0])
    src, dst = moves[HEAD:HEAD + 2 * n].long().view(n, 2).unbind(1)
    s["K"][dst] = s["K"][src]
    s["V"][dst] = s["V"][src]


def _drop(refs, table, gone):
    """The counts without the entries of `table` where `gone`."""
    gone = gone & (table >= 0)
    return refs.scatter_add(0, table.clamp(min=0).reshape(-1), -gone.reshape(-1).long())


def _plain_pages(s):
    case, P, S = s["case"], s["P"], s["case"]["S"]
    s["ints"].copy_(s["ints0"])
    refs, table, lens = s["state"][:P].long(), s["table"].long(), s["lens"].long()
    if case["op"] == "compact":
        live = refs > 0
        L, ids = live.sum(), torch.arange(P, device=refs.device)
        far, hole = live & (ids >= L), ~live & (ids < L)
        holes = torch.sort((~hole).int(), stable=True).indices
        to = torch.where(far, holes[(far.cumsum(0) - 1).clamp(min=0)], ids)
        moves = torch.zeros(HEAD + 2 * s["most"] + 2, dtype=torch.long, device=refs.device)
        slot = torch.where(far, HEAD + 2 * (far.cumsum(0) - 1), HEAD + 2 * s["most"])
        moves[slot], moves[slot + 1] = ids, to
        moves[:HEAD] = torch.stack([far.sum(), far.sum() * 0, L, P - L])
        moves = moves[:HEAD + 2 * s["most"]].int()
        table = torch.where(table >= 0, to[table.clamp(min=0)], -1)
        refs = torch.zeros_like(refs).scatter_add(0, to, refs * live)
        _plain_copy(s, moves)
        return {"refs": refs.int(), "table": table.int(), "moves": moves, "K": s["K"], "V": s["V"]}
    if case["op"] == "fork":
        parent = s["parent"].long()
        new = table[parent]
        refs = refs.scatter_add(0, new.clamp(min=0).reshape(-1), (new >= 0).reshape(-1).long())
        refs = _drop(refs, table, torch.ones_like(table, dtype=torch.bool))
        refs, table, lens, grant, moves = _plain_reserve(refs, new, lens[parent], s["add"].long(), S, case["N"], s["most"])
        _plain_copy(s, moves)
    else:
        left = torch.zeros_like(lens, dtype=torch.bool).index_fill(0, s["leave"].long(), True)
        refs = _drop(refs, table, left[:, None].expand_as(table))
        table, lens = table.masked_fill(left[:, None], -1), lens.masked_fill(left, 0)
        refs, table, lens, grant, moves = _plain_reserve(refs, table, lens, s["count"].long(), S, case["N"], s["most"])
        _put_rows(s["K"], s["k_new"], table, lens, grant)
        _put_rows(s["V"], s["v_new"], table, lens, grant)
    return {"refs": refs.int(), "table": table.int(), "lens": lens.int(), "grant": grant.int(), "moves": moves, "K": s["K"], "V": s["V"]}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "attn":
            return _plain_attn(s)
        if op == "step":
            return _plain_step(s)
        if op == "append":
            table, lens, count = s["table"].long(), s["lens"].long(), s["count"].long()
            _put_rows(s["K"], s["k_new"], table, lens, count)
            _put_rows(s["V"], s["v_new"], table, lens, count)
            return {"K": s["K"], "V": s["V"]}
        return _plain_pages(s)
    from hierarchical_block_sparse_b200 import pisa
    cfg, pages, K, V, table, lens, state = s["cfg"], s["pages"], s["K"], s["V"], s["table"], s["lens"], s["state"]
    if op == "attn":
        new = (s["k_new"], s["v_new"]) if case["append"] else (None, None)
        pisa.pisa_paged_attn(cfg, pages, s["q"], *new, K, V, table, lens, s["o"], s["lse"], s["ws"])
        return {"o": s["o"], "lse": s["lse"], "K": K, "V": V} if case["append"] else {"o": s["o"], "lse": s["lse"]}
    if op == "step":
        pisa.pisa_paged_decode_step(cfg, pages, s["q"], s["k_new"], s["v_new"], K, V, table, lens, s["pyr"], s["idx"], s["o"])
        return {"idx": s["idx"], "o": s["o"], "pyr": s["pyr"]}
    if op == "append":
        pisa.pisa_paged_append(cfg, pages, s["k_new"], s["v_new"], lens, s["count"], table, K, V)
        return {"K": K, "V": V}
    s["ints"].copy_(s["ints0"])
    moves, refs = s["moves"], state[:s["P"]]
    if op == "compact":
        pisa.pisa_pages_compact(cfg, pages, state, table, moves)
        pisa.pisa_pages_copy(cfg, pages, moves, K, V)
        return {"refs": refs, "table": table, "moves": moves, "K": K, "V": V}
    if op == "fork":
        table, lens = s["table_out"], s["lens_out"]
        pisa.pisa_pages_fork(cfg, pages, s["parent"], state, s["table"], s["lens"], table, lens)
        pisa.pisa_pages_reserve(cfg, pages, s["add"], state, table, lens, s["grant"], moves)
        pisa.pisa_pages_copy(cfg, pages, moves, K, V)
    else:
        pisa.pisa_pages_free(cfg, pages, s["leave"], state, table, lens)
        pisa.pisa_pages_reserve(cfg, pages, s["count"], state, table, lens, s["grant"], moves)
        pisa.pisa_paged_append(cfg, pages, s["k_new"], s["v_new"], lens, s["grant"], table, K, V)
    return {"refs": refs, "table": table, "lens": lens, "grant": s["grant"], "moves": moves, "K": K, "V": V}


# ---- from the definitions, in 64 bits ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    n, table = _lens(case), s["table"].cpu().numpy().astype(np.int64)
    op, S, B, Hkv, d = case["op"], case["S"], case["B"], case["Hkv"], case["d"]
    if op in ("attn", "step") and (op == "step" or case["append"]):
        for b in range(B):
            if n[b] > 0:
                t = int(n[b]) - 1
                s["K"][table[b, t // S], :, t % S], s["V"][table[b, t // S], :, t % S] = s["k_new"][b], s["v_new"][b]
    if op == "attn":
        return _exact_attn(s, n, table)
    if op == "step":
        return _exact_step(s, n, table)
    if op == "append":
        _exact_put(s, n, _counts(case), table)
        return {"K": s["K"], "V": s["V"]}
    return _exact_pages(s, n, table)


def _sequence(pool, row, n, S):
    """The first n rows of one sequence in 64 bits: [Hkv, n, d]."""
    ids = torch.from_numpy(row[: -(-n // S)]).to(pool.device)
    return torch.cat(list(pool[ids].unbind(0)), 1)[:, :n].double()


def _exact_attn(s, n, table):
    case = s["case"]
    Hq, Hkv, d, S = (case[k] for k in ("Hq", "Hkv", "d", "S"))
    o = torch.zeros(case["B"], Hq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((case["B"], Hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for b in range(case["B"]):
        if n[b] == 0:
            continue
        k, v = _sequence(s["K"], table[b], int(n[b]), S), _sequence(s["V"], table[b], int(n[b]), S)
        q = s["q"][b].double().view(Hkv, Hq // Hkv, d)
        z = torch.einsum("hgd,hnd->hgn", q, k) * d ** -0.5
        lse[b] = torch.logsumexp(z, -1).view(Hq)
        o[b] = torch.einsum("hgn,hnd->hgd", torch.exp(z - lse[b].view(Hkv, -1, 1)), v).reshape(Hq, d)
    out = {"o": o, "lse": lse}
    return dict(out, K=s["K"], V=s["V"]) if case["append"] else out


def _exact_step(s, n, table):
    """Every node of every level is scored; the walk then takes its choices from that."""
    case = s["case"]
    B, Hq, Hkv, d, S, C, K = (case[k] for k in ("B", "Hq", "Hkv", "d", "S", "C", "K"))
    dev, G = s["q"].device, Hq // Hkv
    idx = np.full((B, Hkv, K), -1, np.int32)
    o = torch.zeros(B, Hq, d, dtype=torch.float64, device=dev)
    levels, off = _levels(case["N"], C)
    pyr = torch.zeros(B, Hkv, off[-1] + levels[-1], d, dtype=torch.float64, device=dev)
    for b in range(B):
        t = int(n[b]) - 1
        k, v = _sequence(s["K"], table[b], t + 1, S), _sequence(s["V"], table[b], t + 1, S)
        q = s["q"][b].double().view(Hkv, G, d)
        z = torch.einsum("hgd,hnd->hgn", q, k) * d ** -0.5
        scores = []
        for lv in range(len(levels)):
            if lv == 0:
                rows = torch.stack([k[:, i:i + C].mean(1) for i in range(0, t + 1, C)], 1)
                parts, each = z, C
            else:
                parts, each = torch.einsum("hgd,hmd->hgm", q, rows) * d ** -0.5, 2
                rows = torch.stack([rows[:, i:i + 2].mean(1) for i in range(0, rows.shape[1], 2)], 1)
            pad = torch.nn.functional.pad(parts, (0, -parts.shape[-1] % each), value=-math.inf)
            scores.append(torch.logsumexp(pad.view(Hkv, G, -1, each), -1).sum(1).cpu().numpy())
            pyr[b, :, off[lv]:off[lv] + rows.shape[1]] = rows
        last = t // C
        for h in range(Hkv):
            nodes = [0]
            for lv in range(len(levels) - 1, -1, -1):
                nodes = [x for x in nodes if x < scores[lv].shape[1]]
                must = {0, last >> lv} | ({(last - 1) >> lv} if last else set())
                if len(nodes) > K:
                    nodes = sorted(nodes, key=lambda x: (x not in must, -scores[lv][h, x], x))[:K]
                nodes = sorted(nodes)
                kept = nodes
                nodes = [c for x in nodes for c in (2 * x, 2 * x + 1)]
            idx[b, h, :len(kept)] = kept
            cols = torch.tensor([j for x in kept for j in range(x * C, min(x * C + C, t + 1))], device=dev)
            p = torch.softmax(z[h][:, cols], -1)
            o[b, h * G:(h + 1) * G] = p @ v[h, cols]
    return {"idx": torch.from_numpy(idx), "o": o, "pyr": pyr}


def _exact_put(s, n, count, table):
    S = s["case"]["S"]
    for b in range(s["case"]["B"]):
        i, c = 0, int(count[b])
        while i < c:  # one page at a time
            t = int(n[b]) - c + i
            m = min(c - i, S - t % S)
            for pool, rows in ((s["K"], s["k_new"]), (s["V"], s["v_new"])):
                pool[table[b, t // S], :, t % S:t % S + m] = rows[b, :, i:i + m]
            i += m


def _exact_pages(s, n, table):
    """The page calls told one sequence and one page after another."""
    case, P, S, B = s["case"], s["P"], s["case"]["S"], s["case"]["B"]
    refs, n = s["state"][:P].cpu().numpy().copy(), n.copy()
    moves, pairs, missing = np.zeros(HEAD + 2 * s["most"], np.int32), [], 0
    grant = np.zeros(B, np.int32)
    if case["op"] == "compact":
        L = int((refs > 0).sum())
        holes = [i for i in range(L) if refs[i] == 0]
        pairs = list(zip([i for i in range(L, P) if refs[i] > 0], holes))
        for a, z in pairs:
            refs[z], refs[a] = refs[a], 0
        to = dict(pairs)
        table = np.array([[to.get(x, x) for x in row] for row in table.tolist()], np.int64).reshape(table.shape)
    else:
        if case["op"] == "fork":
            parent = s["parent"].cpu().numpy()
            old, table, n, add = table, table[parent], n[parent], s["add"].cpu().numpy()
            for x in table[table >= 0]:
                refs[x] += 1
            for x in old[old >= 0]:
                refs[x] -= 1
        else:
            add = s["count"].cpu().numpy()
            for b in s["leave"].tolist():
                for x in table[b][table[b] >= 0]:
                    refs[x] -= 1
                table[b], n[b] = -1, 0
        free = [i for i in range(P) if refs[i] == 0]
        before, need, plan = refs.copy(), 0, []
        for b in range(B):
            a = int(add[b])
            if a <= 0 or n[b] + a > case["N"]:
                continue
            have, want = -(-int(n[b]) // S), -(-int(n[b] + a) // S)
            ids = list(range(have, want))
            if n[b] % S and before[table[b, have - 1]] > 1:
                before[table[b, have - 1]] -= 1
                ids = [have - 1] + ids
            plan.append((b, a, ids))
            need += len(ids)
        if need <= len(free):
            for b, a, ids in plan:
                for w in ids:
                    page = free.pop(0)
                    if table[b, w] >= 0:
                        pairs.append((int(table[b, w]), page))
                        refs[table[b, w]] -= 1
                    table[b, w], refs[page] = page, 1
                grant[b], n[b] = a, n[b] + a
        else:
            missing = need - len(free)
    live = int((refs > 0).sum())
    moves[:HEAD] = [len(pairs), missing, live, P - live]
    if pairs:
        moves[HEAD:HEAD + 2 * len(pairs)] = np.array(pairs, np.int32).reshape(-1)
    if case["op"] != "admit" and pairs:
        src, dst = (torch.tensor(x, device=s["K"].device) for x in zip(*pairs))
        s["K"][dst], s["V"][dst] = s["K"][src].clone(), s["V"][src].clone()
    if case["op"] == "admit":
        _exact_put(s, n, grant, table)
    out = {"refs": torch.from_numpy(refs.astype(np.int32)), "table": torch.from_numpy(table.astype(np.int32)),
           "moves": torch.from_numpy(moves), "K": s["K"], "V": s["V"]}
    if case["op"] != "compact":
        out.update(lens=torch.from_numpy(n.astype(np.int32)), grant=torch.from_numpy(grant))
    return out
