"""Workloads of the paged key/value cache: attention of new tokens over pages,
and the operators that hand out, share, move and drop pages.

Each case is one call (or one pair of calls) that a serving program makes.
`run` computes it in plain torch operations, or, with `own`, through
gated_linear_sliding_chunkwise_b200.paged.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one user, one token, a short context: what a call costs
        dict(name="attn_one_token", op="attn", dtype="bf16", B=1, H=32, Hkv=8, d=128, page=64, new_lo=1, new_hi=1,
             chunks=0, len_lo=517, len_hi=517, window=0, sinks=0),
        # a full decode batch of mixed ages over long contexts
        dict(name="attn_decode_batch", op="attn", dtype="bf16", B=64, H=32, Hkv=8, d=128, page=64, new_lo=1, new_hi=1,
             chunks=0, len_lo=1000, len_hi=16384, window=0, sinks=0),
        # continuous batching: decoding users and a few prompt chunks in one call,
        # seven query heads to a kv head, a window with four first tokens kept
        dict(name="attn_mixed_window", op="attn", dtype="bf16", B=48, H=14, Hkv=2, d=64, page=16, new_lo=1, new_hi=255,
             chunks=4, len_lo=300, len_hi=9001, window=1024, sinks=4),
        # prompt chunks of four users
        dict(name="attn_chunks", op="attn", dtype="bf16", B=4, H=32, Hkv=8, d=128, page=128, new_lo=77, new_hi=512,
             chunks=4, len_lo=1500, len_hi=8191, window=0, sinks=0),
        # the second half of a 16K-token prompt
        dict(name="attn_long_prompt", op="attn", dtype="bf16", B=1, H=32, Hkv=8, d=128, page=64, new_lo=8192,
             new_hi=8192, chunks=1, len_lo=16384, len_hi=16384, window=0, sinks=0),
        # fp32 activations, as the parity runs use them
        dict(name="attn_chunks_fp32", op="attn", dtype="fp32", B=2, H=8, Hkv=8, d=64, page=32, new_lo=150, new_hi=233,
             chunks=2, len_lo=700, len_hi=1501, window=0, sinks=0),
        # one prompt answered four ways
        dict(name="fork_one_prompt", op="fork", dtype="bf16", layers=4, pages=256, Hkv=8, d=128, page=64, parents=1,
             children=4, len_lo=1000, len_hi=1000),
        # beam or group sampling: 24 prompts, eight branches each
        dict(name="fork_many", op="fork", dtype="bf16", layers=16, pages=1200, Hkv=8, d=128, page=64, parents=24,
             children=8, len_lo=200, len_hi=2000),
        # one user leaves and another arrives
        dict(name="turnover_one", op="turnover", pages=2048, page=64, rows=16, turn=1, len_lo=100, len_hi=4000),
        # many users leave and arrive in a large pool of small pages
        dict(name="turnover_many", op="turnover", pages=131072, page=16, rows=512, turn=256, len_lo=100, len_hi=6000),
        # a small fp32 pool closed up
        dict(name="compact_small", op="compact", dtype="fp32", layers=2, pages=96, Hkv=4, d=64, page=16, live=0.4),
        # a fragmented pool closed up before half of it is given back
        dict(name="compact_pool", op="compact", dtype="bf16", layers=16, pages=1000, Hkv=8, d=128, page=64, live=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "fork", "turnover", "compact"])
    if op == "attn":
        d = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 3, 4, 5, 7, 8])
        page = rng.choice([16, 32, 64, 128])
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 16, 4096), 0), (_log(rng, 16, 4096), rng.randint(1, 200))])
        if rng.random() < 0.5:   # decoding, or a few tokens at a time
            B, hi, new = _log(rng, 1, 64), _log(rng, 64, 16384), rng.choice([1, 1, 2, rng.randint(3, 9)])
            if dtype == "fp32":
                B, hi = min(B, 16), min(hi, 4096)
            return dict(op=op, dtype=dtype, B=B, H=Hkv * g, Hkv=Hkv, d=d, page=page, new_lo=1, new_hi=new, chunks=B,
                        len_lo=max(new, hi // 16), len_hi=hi, window=window, sinks=sinks)
        B = _log(rng, 1, 24)
        hi = _log(rng, 256, 8192 if B < 5 else 4096)
        if dtype == "fp32":
            hi = min(hi, 2048)
        new = min(hi, _log(rng, 10, 2000 if B < 5 else 300))
        return dict(op=op, dtype=dtype, B=B, H=Hkv * g, Hkv=Hkv, d=d, page=page, new_lo=max(1, new // 8), new_hi=new,
                    chunks=rng.randint(1, B), len_lo=max(new, hi // 8), len_hi=hi, window=window, sinks=sinks)
    if op == "turnover":
        rows = _log(rng, 2, 512)
        page = rng.choice([16, 32, 64, 128])
        hi = _log(rng, 60, 6000)
        turn = rng.randint(1, max(1, rows // 2))
        pages = (rows + turn) * (hi // page + 1) + rng.randint(0, 500)
        return dict(op=op, pages=pages, page=page, rows=rows, turn=turn, len_lo=max(1, hi // 20), len_hi=hi)
    layers = rng.choice([1, 2, 3, 8, 16])
    Hkv, d, page = rng.choice([1, 2, 4, 8]), rng.choice([64, 128]), rng.choice([16, 32, 64])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "fork":
        parents, children, hi = _log(rng, 1, 24), rng.randint(1, 8), _log(rng, 20, 1000)
        pages = parents * (hi // page + 1) + 3 * parents * children + rng.randint(0, 60)
        return dict(op=op, dtype=dtype, layers=layers, pages=pages, Hkv=Hkv, d=d, page=page, parents=parents,
                    children=children, len_lo=max(1, hi // 8), len_hi=hi)
    return dict(op=op, dtype=dtype, layers=layers, pages=_log(rng, 20, 900), Hkv=Hkv, d=d, page=page,
                live=rng.uniform(0.1, 0.9))


# ------------------------------------------------------------------ inputs
def _plan(case):
    """The call's host-side numbers: tokens and lengths of each sequence.  They
    follow from the sizes of the case alone, spread evenly over its ranges."""
    B, chunks = case["B"], case["chunks"]
    new, lens = [], []
    for b in range(B):
        f = (b * 0.6180339887) % 1.0           # a fixed spread over the ranges
        big = b >= B - chunks
        lo, hi = case["new_lo"], case["new_hi"]
        n = lo + int(round((hi - lo) * (1.0 if b == B - 1 else f))) if big else lo
        s = case["len_lo"] + int(round((case["len_hi"] - case["len_lo"]) * (1.0 if b == B - 1 else f)))
        new.append(n)
        lens.append(max(s, n))
    return new, lens


def _ceil(a, b):
    return -(-a // b)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = torch.device("cuda")

    def normal(*shape, dtype):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    op, page = case["op"], case["page"]
    if op == "attn":
        dt = DTYPES[case["dtype"]]
        new, lens = _plan(case)
        H, Hkv, d = case["H"], case["Hkv"], case["d"]
        T, used = sum(new), [_ceil(s, page) for s in lens]
        P, MP = sum(used) + 3, max(used)
        perm = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
        col = torch.arange(MP, device=dev)
        u = torch.tensor(used, device=dev)
        first = torch.cumsum(u, 0) - u
        # a sequence's pages lie anywhere in the pool; unused entries are -1
        table = torch.where(col < u[:, None], perm[(first[:, None] + col).clamp(max=P - 1)], -1).to(torch.int32)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        return dict(case=case, q=normal(T, H, d, dtype=dt), k=normal(T, Hkv, d, dtype=dt),
                    v=normal(T, Hkv, d, dtype=dt), k_pages=normal(1, P, Hkv, page, d, dtype=dt),
                    v_pages=normal(1, P, Hkv, page, d, dtype=dt), table=table.contiguous(), lens=ints(lens),
                    cu_q=ints(cu), max_q=max(new), max_len=max(lens), new=new, ctx=lens)
    if op == "turnover":
        P, R, n = case["pages"], case["rows"], case["turn"]
        span = case["len_hi"] - case["len_lo"]
        lens = case["len_lo"] + torch.randint(0, span + 1, (R,), generator=gen, device=dev)
        grow = case["len_lo"] + torch.randint(0, span + 1, (n,), generator=gen, device=dev)
        rows = torch.randperm(R, generator=gen, device=dev)[:n]
        refs, table = _rows_of_pool(lens, P, page, _ceil(case["len_hi"], page), gen)
        return dict(case=case, refs=refs, table=table, lens=lens.to(torch.int32), rows=rows.to(torch.int32),
                    grow=grow.to(torch.int32))
    dt = DTYPES[case["dtype"]]
    P = case["pages"]
    shape = (case["layers"], P, case["Hkv"], page, case["d"])
    k_pages, v_pages = normal(*shape, dtype=dt), normal(*shape, dtype=dt)
    if op == "fork":
        n, c = case["parents"], case["children"]
        R = n * (c + 1)
        lens = torch.zeros(R, dtype=torch.int64, device=dev)
        span = case["len_hi"] - case["len_lo"]
        plen = case["len_lo"] + torch.randint(0, span + 1, (n,), generator=gen, device=dev)
        lens[:n] = plen
        refs, table = _rows_of_pool(lens, P, page, _ceil(case["len_hi"], page), gen)
        src = torch.arange(n, device=dev).repeat_interleave(c)
        dst = torch.arange(n, R, device=dev)
        return dict(case=case, k_pages=k_pages, v_pages=v_pages, refs=refs, table=table, lens=lens.to(torch.int32),
                    src=src.to(torch.int32), dst=dst.to(torch.int32))
    # compact: rows of 8 entries over live pages scattered in the pool
    live = max(1, min(P - 1, int(round(case["live"] * P))))
    perm = torch.randperm(P, generator=gen, device=dev)[:live].to(torch.int32)
    refs = torch.zeros(P, dtype=torch.int32, device=dev)
    refs[perm.long()] = 1
    R = _ceil(live, 8) + 1                     # the last row shares the first row's pages
    table = torch.full((R * 8,), -1, dtype=torch.int32, device=dev)
    table[:live] = perm
    shared = min(8, live)
    table[(R - 1) * 8:(R - 1) * 8 + shared] = perm[:shared]
    refs[perm[:shared].long()] += 1
    return dict(case=case, k_pages=k_pages, v_pages=v_pages, refs=refs, table=table.view(R, 8).contiguous())


def _rows_of_pool(lens, P, page, MP, gen):
    """Counts and table of rows of these lengths over random pages of the pool."""
    dev = lens.device
    used = (lens + page - 1) // page
    first = torch.cumsum(used, 0) - used
    perm = torch.randperm(P, generator=gen, device=dev).to(torch.int32)
    col = torch.arange(MP, device=dev)
    hold = col < used[:, None]
    table = torch.where(hold, perm[(first[:, None] + col).clamp(max=P - 1)], -1).to(torch.int32)
    refs = torch.zeros(P, dtype=torch.int32, device=dev)
    refs[table[hold].long()] = 1
    return refs, table.contiguous()


# -------------------------------------------------------------- plain forms
def _plain_attn(s):
    c = s["case"]
    page, H, Hkv, d = c["page"], c["H"], c["Hkv"], c["d"]
    g, dev = H // Hkv, s["q"].device
    lens, cu, table = s["lens"].long(), s["cu_q"].long(), s["table"].long()
    new = cu[1:] - cu[:-1]
    T, N, S = s["q"].shape[0], s["max_q"], s["max_len"]
    # the new tokens go into their pages
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu, t, right=True) - 1
    at = lens[b] - new[b] + t - cu[b]
    pid = table[b, at // page]
    s["k_pages"][0][pid, :, at % page] = s["k"]
    s["v_pages"][0][pid, :, at % page] = s["v"]
    # every sequence's keys and values, padded to the longest
    ids = table[:, : _ceil(S, page)].clamp(min=0)
    K = s["k_pages"][0][ids].transpose(1, 2).reshape(len(lens), Hkv, -1, d)[:, :, :S].float()
    V = s["v_pages"][0][ids].transpose(1, 2).reshape(len(lens), Hkv, -1, d)[:, :, :S].float()
    i = torch.arange(N, device=dev)
    Q = s["q"][(cu[:-1, None] + i).clamp(max=T - 1)].float()                  # [B, N, H, d]
    Q = Q.view(-1, N, Hkv, g, d).permute(0, 2, 3, 1, 4).reshape(-1, Hkv, g * N, d)
    p = (lens - new)[:, None] + i                                             # position of each new token
    j = torch.arange(S, device=dev)
    see = j <= p[..., None]
    if c["window"]:
        see &= (j > p[..., None] - c["window"]) | (j < c["sinks"])
    x = (Q @ K.transpose(2, 3)).view(-1, Hkv, g, N, S)
    x *= 1.0 / math.sqrt(d)
    x.masked_fill_(~see[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    x -= m
    x.exp_()
    l = x.sum(-1, keepdim=True)
    o = (x.view(-1, Hkv, g * N, S) @ V).view(-1, Hkv, g, N, d) / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + l.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4)[b, t - cu[b]].reshape(T, H, d).to(s["q"].dtype)
    lse = lse.permute(0, 3, 1, 2)[b, t - cu[b]].reshape(T, H)
    return dict(o=o, lse=lse, k_pages=s["k_pages"], v_pages=s["v_pages"])


def _free_pages(refs):
    """Page numbers, the free ones first, each kind in ascending order."""
    return torch.sort((refs != 0).to(torch.int32), stable=True).indices


def _plain_free(s):
    page, rows = s["case"]["page"], s["rows"].long()
    held = (s["lens"][rows] + page - 1) // page
    ids = s["table"][rows]
    hold = torch.arange(ids.shape[1], device=ids.device) < held[:, None]
    s["refs"].index_add_(0, ids.clamp(min=0).flatten().long(), -hold.flatten().to(torch.int32))
    s["table"][rows] = -1
    s["lens"][rows] = 0


def _plain_reserve(s):
    page, rows = s["case"]["page"], s["rows"].long()
    old = s["lens"][rows]
    had, has = (old + page - 1) // page, (old + s["grow"] + page - 1) // page
    need = has - had
    first = torch.cumsum(need, 0) - need
    ids = _free_pages(s["refs"])
    taken = torch.arange(len(ids), device=ids.device) < need.sum()
    col = torch.arange(s["table"].shape[1], device=ids.device)
    fresh = (col >= had[:, None]) & (col < has[:, None])
    pick = ids[(first[:, None] + col - had[:, None]).clamp(0, len(ids) - 1)].to(torch.int32)
    s["table"][rows] = torch.where(fresh, pick, s["table"][rows])
    s["refs"][ids] += taken.to(torch.int32)
    s["lens"][rows] = old + s["grow"]


def _plain_fork(s):
    page, src, dst = s["case"]["page"], s["src"].long(), s["dst"].long()
    refs, table, lens = s["refs"], s["table"], s["lens"]
    ids, n, old, held = table[src], lens[src], table[dst], (lens[dst] + page - 1) // page
    part = (n % page != 0) & (src != dst)
    move = (src != dst)[:, None]
    col = torch.arange(ids.shape[1], device=ids.device)
    tail = n // page
    new = _free_pages(refs)[(torch.cumsum(part, 0) - 1).clamp(min=0)].to(torch.int32)
    is_tail = part[:, None] & (col == tail[:, None])
    # the part-filled last page of each source is copied, in every layer; a row without one copies its first page to itself
    frm = torch.where(part, ids.gather(1, tail.clamp(max=ids.shape[1] - 1)[:, None].long())[:, 0], ids[:, 0]).long()
    to = torch.where(part, new, ids[:, 0]).long()
    s["k_pages"][:, to] = s["k_pages"][:, frm]
    s["v_pages"][:, to] = s["v_pages"][:, frm]
    out = torch.where(is_tail, new[:, None], ids)
    out = torch.where(move, out, old)
    up = move & (col < ((n + page - 1) // page)[:, None])
    down = move & (col < held[:, None])
    refs.index_add_(0, out.clamp(min=0).flatten().long(), up.flatten().to(torch.int32))
    refs.index_add_(0, old.clamp(min=0).flatten().long(), -down.flatten().to(torch.int32))
    table[dst] = out
    lens[dst] = torch.where(src != dst, n, lens[dst])


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    P = refs.shape[0]
    live = refs > 0
    L = live.sum()
    at = torch.arange(P, device=refs.device)
    frm, to = (live & (at >= L)).nonzero()[:, 0], (~live & (at < L)).nonzero()[:, 0]
    s["k_pages"][:, to] = s["k_pages"][:, frm]
    s["v_pages"][:, to] = s["v_pages"][:, frm]
    place = at.clone()
    place[frm] = to
    table_out = torch.where(table >= 0, place[table.clamp(min=0).long()].to(torch.int32), table)
    refs_out = refs.clone()
    refs_out[to] = refs[frm]
    refs_out[frm] = 0
    return table_out, refs_out


def run(state):
    s, c = state, state["case"]
    if own:
        from gated_linear_sliding_chunkwise_b200 import paged
    if c["op"] == "attn":
        if own:
            r = paged.attn(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu_q"],
                           max_q=s["max_q"], window=c["window"], sinks=c["sinks"], want_lse=True)
            return dict(o=r["o"], lse=r["lse"], k_pages=s["k_pages"], v_pages=s["v_pages"])
        return _plain_attn(s)
    if c["op"] == "turnover":                  # users leave, others take their rows
        if own:
            paged.free(s["refs"], s["table"], s["lens"], s["rows"], page=c["page"])
            paged.reserve(s["refs"], s["table"], s["lens"], s["rows"], s["grow"], page=c["page"])
        else:
            _plain_free(s)
            _plain_reserve(s)
        return dict(refs=s["refs"], table=s["table"], lens=s["lens"])
    if c["op"] == "fork":
        if own:
            paged.fork(s["k_pages"], s["v_pages"], s["refs"], s["table"], s["lens"], s["src"], s["dst"])
        else:
            _plain_fork(s)
        return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], refs=s["refs"], table=s["table"], lens=s["lens"])
    if own:
        table, refs = paged.compact(s["k_pages"], s["v_pages"], s["refs"], s["table"])
    else:
        table, refs = _plain_compact(s)
    return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], refs=refs, table=table)


# --------------------------------------------------------------------- work
def _pairs(n, s, window, sinks):
    """(Visible pairs of n new tokens that end a sequence of s, keys that any of them sees.)"""
    total = 0
    for p in range(s - n, s):
        seen = p + 1
        if window:
            lo = max(0, p - window + 1)
            seen = p + 1 - lo + min(sinks, lo)
        total += seen
    keys = s
    if window:
        lo = max(0, s - n - window + 1)
        keys = s - lo + min(sinks, lo)
    return total, keys


def work(case):
    op, page = case["op"], case["page"]
    if op == "turnover":
        # counts read and those of the pages that change hands written, two rows of the table for each user
        entries = case["turn"] * _ceil((case["len_lo"] + case["len_hi"]) // 2, page)
        return dict(bytes=4.0 * (case["pages"] + 6 * entries + 6 * case["turn"]), flops=0.0)
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "attn":
        new, lens = _plan(case)
        pairs = keys = 0
        for n, s in zip(new, lens):
            a, b = _pairs(n, s, case["window"], case["sinks"])
            pairs, keys = pairs + a, keys + b
        T, d = sum(new), case["d"]
        kv = 2 * case["Hkv"] * d * e
        return dict(bytes=float(2 * T * case["H"] * d * e + 4 * T * case["H"] + 2 * T * kv + (keys - T) * kv),
                    flops=4.0 * d * case["H"] * pairs)
    size = 2 * case["layers"] * case["Hkv"] * page * case["d"] * e       # one page, K and V, every layer
    if op == "fork":
        n = case["parents"] * case["children"]
        avg = (case["len_lo"] + case["len_hi"]) // 2
        # children of one prompt copy the same page: it is read once
        return dict(bytes=float((n + case["parents"]) * size + 4 * (case["pages"] + 3 * n * _ceil(avg, page))), flops=0.0)
    P, live = case["pages"], case["live"]
    moved = live * (1 - live) * P                                         # expected
    return dict(bytes=float(2 * moved * size + 4 * (2 * P + 2 * live * P)), flops=0.0)


# ------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, page = case["op"], case["page"]
    if op == "attn":
        return _exact_attn(case, s)
    refs, table = s["refs"].tolist(), s["table"].tolist()
    dev = s["refs"].device

    def whole(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    if op == "compact":
        P = len(refs)
        L = sum(r > 0 for r in refs)
        frm, to = [p for p in range(L, P) if refs[p] > 0], [p for p in range(L) if refs[p] == 0]
        place = dict(zip(frm, to))
        for a, b in place.items():
            refs[b], refs[a] = refs[a], 0
            for pool in (s["k_pages"], s["v_pages"]):
                pool[:, b].copy_(pool[:, a])
        return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], refs=whole(refs),
                    table=whole([[place.get(p, p) for p in row] for row in table]))
    lens = s["lens"].tolist()
    if op == "turnover":
        for r in s["rows"].tolist():
            for j in range(_ceil(lens[r], page)):
                refs[table[r][j]] -= 1
            table[r], lens[r] = [-1] * len(table[r]), 0
        spare = iter([p for p, r in enumerate(refs) if r == 0])
        for r, n in zip(s["rows"].tolist(), s["grow"].tolist()):
            for j in range(_ceil(n, page)):
                table[r][j] = next(spare)
                refs[table[r][j]] = 1
            lens[r] = n
        return dict(refs=whole(refs), table=whole(table), lens=whole(lens))
    spare = iter([p for p, r in enumerate(refs) if r == 0])
    before, length = [list(r) for r in table], list(lens)
    pairs = [(a, b) for a, b in zip(s["src"].tolist(), s["dst"].tolist()) if a != b]
    for a, b in pairs:
        row = list(before[a])
        if length[a] % page:
            j = length[a] // page
            row[j] = next(spare)
            for pool in (s["k_pages"], s["v_pages"]):
                pool[:, row[j]].copy_(pool[:, before[a][j]])
        for j in range(_ceil(length[a], page)):
            refs[row[j]] += 1
        table[b], lens[b] = row, length[a]
    for _, b in pairs:
        for j in range(_ceil(length[b], page)):
            refs[before[b][j]] -= 1
    return dict(k_pages=s["k_pages"], v_pages=s["v_pages"], refs=whole(refs), table=whole(table), lens=whole(lens))


def _exact_attn(case, s):
    page, H, Hkv, d = case["page"], case["H"], case["Hkv"], case["d"]
    g, dev = H // Hkv, s["q"].device
    T = s["q"].shape[0]
    o = torch.zeros(T, H, d, dtype=torch.float64, device=dev)
    lse = torch.zeros(T, H, dtype=torch.float64, device=dev)
    t0 = 0
    for b, (n, ctx) in enumerate(zip(s["new"], s["ctx"])):
        pos = torch.arange(ctx, device=dev)
        pid, off = s["table"][b].long()[pos // page], pos % page
        for pool, x in ((s["k_pages"], s["k"]), (s["v_pages"], s["v"])):
            pool[0].index_put_((pid[ctx - n:], torch.arange(Hkv, device=dev)[:, None], off[ctx - n:]),
                               x[t0:t0 + n].transpose(0, 1))
        for h in range(Hkv):
            k = s["k_pages"][0, pid, h, off].double()
            v = s["v_pages"][0, pid, h, off].double()
            step = max(1, (1 << 28) // (ctx * g))                           # query rows at a time
            for a in range(0, n, step):
                z = min(n, a + step)
                p = torch.arange(ctx - n + a, ctx - n + z, device=dev)[:, None]
                hide = pos[None] > p
                if case["window"]:
                    hide |= (pos[None] <= p - case["window"]) & (pos[None] >= case["sinks"])
                x = torch.einsum("ngd,sd->ngs", s["q"][t0 + a:t0 + z, h * g:(h + 1) * g].double(), k) / math.sqrt(d)
                x = x.masked_fill(hide[:, None], -math.inf)
                lse[t0 + a:t0 + z, h * g:(h + 1) * g] = torch.logsumexp(x, -1)
                o[t0 + a:t0 + z, h * g:(h + 1) * g] = torch.softmax(x, -1) @ v
        t0 += n
    return dict(o=o, lse=lse, k_pages=s["k_pages"], v_pages=s["v_pages"])
