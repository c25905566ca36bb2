"""Plain 64-bit model of the paged cache, shared by its tests: attention over
the pages, and the bookkeeping on Python lists."""

import math

import torch


def ceil_div(a, b):
    return -(-a // b)


def build(seqs, *, Hkv, d, page, dtype, layers=1, spare=3, seed=0, fill=0.0, max_pages=None):
    """A cache whose row b holds seqs[b] tokens on random pages; slots and
    pages that hold no token are filled with `fill`.  CPU tensors."""
    gen = torch.Generator().manual_seed(seed)
    used = [ceil_div(s, page) for s in seqs]
    P = sum(used) + spare
    MP = max(max(used), 1) if max_pages is None else max_pages
    perm = torch.randperm(P, generator=gen).tolist()
    table = torch.full((len(seqs), MP), -1, dtype=torch.int32)
    k = torch.full((layers, P, Hkv, page, d), fill, dtype=dtype)
    v = torch.full_like(k, fill)
    refs = torch.zeros(P, dtype=torch.int32)
    at = 0
    for b, s in enumerate(seqs):
        for j in range(used[b]):
            p = perm[at]
            at += 1
            table[b, j] = p
            refs[p] = 1
            n = min(page, s - j * page)
            k[:, p, :, :n] = torch.randn(layers, Hkv, n, d, generator=gen).to(dtype)
            v[:, p, :, :n] = torch.randn(layers, Hkv, n, d, generator=gen).to(dtype)
    return dict(k_pages=k, v_pages=v, table=table, lens=torch.tensor(seqs, dtype=torch.int32), refs=refs)


def gather(pool, table_row, n, page):
    """[Hkv, n, d] fp64: tokens 0 .. n - 1 of a row of one layer's pool."""
    t = torch.arange(n)
    return pool[table_row.long()[t // page], :, t % page].permute(1, 0, 2).double()


def attention(q, k_pages, v_pages, table, lens, cu, *, window=0, sinks=0, scale=None, row=None):
    """fp64 o, lse and A = sum_j p_j |v_j| (the scale of o's error), and the
    largest sum |q_i k_i| of a visible pair times the scale, per (token, head).
    Tokens of no sequence stay NaN."""
    T, H, d = q.shape
    Hkv, page = k_pages.shape[1], k_pages.shape[2]
    g = H // Hkv
    scale = scale or 1.0 / math.sqrt(d)
    o = torch.full((T, H, d), math.nan, dtype=torch.float64)
    A = torch.zeros(T, H, d, dtype=torch.float64)
    lse = torch.full((T, H), math.nan, dtype=torch.float64)
    mag = torch.zeros(T, H, dtype=torch.float64)
    cu = cu.tolist()
    for b in range(len(cu) - 1):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        r = b if row is None else int(row[b])
        s = int(lens[r])
        K, V = gather(k_pages, table[r], s, page), gather(v_pages, table[r], s, page)
        for i in range(n):
            p = s - n + i
            seen = [j for j in range(p + 1) if window == 0 or j > p - window or j < sinks]
            t = cu[b] + i
            if not seen:
                o[t], lse[t] = 0.0, -math.inf
                continue
            for h in range(H):
                kk, vv = K[h // g][seen], V[h // g][seen]
                x = (kk @ q[t, h].double()) * scale
                m = x.max()
                w = (x - m).exp()
                lse[t, h] = m + w.sum().log()
                w = w / w.sum()
                o[t, h] = w @ vv
                A[t, h] = w @ vv.abs()
                mag[t, h] = (kk.abs() @ q[t, h].double().abs()).max() * scale
    return o, lse, A, mag


def check_attention(name, got_o, got_lse, want, d, dtype, rounded_weights):
    """Element by element against the error that the arithmetic allows.

    Logits: d products summed in 32 bits, each step off by at most 2^-22 of the
    running magnitude (a tensor core may cut where an FMA rounds): delta =
    (d + 4) 2^-22 sum |q_i k_i| scale.  A weight is then off by a factor within
    exp(+-2 delta) (its own logit and the normaliser's), plus 2^-20 for exp2,
    the sums and the division; rounded to bf16 it is off by another half step,
    2^-8, while the normaliser sums what was not rounded.  So |o - want| <=
    A (2 delta + 2^-20 [+ 2^-8]), A = sum_j p_j |v_j|; then o's own rounding."""
    o, lse, A, mag = want
    live = ~torch.isnan(lse)
    delta = (d + 4) * 2.0 ** -22 * mag
    weight = 2.0 ** -8 if rounded_weights else 0.0
    tol = A * (2.0 * delta + 2.0 ** -20 + weight).unsqueeze(-1)
    half = torch.finfo(dtype).eps / 2
    tol = tol * (1 + half) + half * o.abs() + 1e-30
    err = (got_o.double().cpu() - o).abs()
    bad = (err > tol) & live.unsqueeze(-1)
    assert torch.isfinite(got_o.double().cpu()[live]).all(), f"{name}: not finite"
    worst = float((err / tol)[live].max()) if live.any() else 0.0
    print(f"PAGED {name} worst error / bound {worst:.3f}")
    assert not bad.any(), f"{name}: {int(bad.sum())} elements outside the bound, worst {worst:.2f} of it"
    if got_lse is not None:
        got = got_lse.double().cpu()
        empty = live & torch.isinf(lse)
        assert torch.equal(got[empty], lse[empty]), f"{name}: lse of rows without keys"
        some = live & ~torch.isinf(lse)
        ltol = delta + 2.0 ** -20 + lse.abs() * 2.0 ** -23
        lerr = (got - lse).abs()
        assert (lerr[some] <= ltol[some]).all(), f"{name}: lse off by {float((lerr / ltol)[some].max()):.2f} of its bound"


class Model:
    """The bookkeeping on lists.  `contents[p]` names what page p holds."""

    def __init__(self, refs, table, lens, page):
        self.refs, self.table = refs.tolist(), table.tolist()
        self.lens, self.page = lens.tolist(), page
        self.contents = list(range(len(self.refs)))

    def _free(self):
        return iter([p for p, r in enumerate(self.refs) if r == 0])

    def _held(self, r):
        return ceil_div(self.lens[r], self.page)

    def reserve(self, rows, grow):
        spare = self._free()
        for r, g in zip(rows, grow):
            for j in range(self._held(r), ceil_div(self.lens[r] + g, self.page)):
                self.table[r][j] = next(spare)
                self.refs[self.table[r][j]] = 1
            self.lens[r] += g

    def free(self, rows):
        for r in rows:
            for j in range(self._held(r)):
                self.refs[self.table[r][j]] -= 1
            self.table[r] = [-1] * len(self.table[r])
            self.lens[r] = 0

    def fork(self, src, rows):
        spare = self._free()
        table, lens, contents = [list(x) for x in self.table], list(self.lens), list(self.contents)
        pairs = [(a, b) for a, b in zip(src, rows) if a != b]
        for _, b in pairs:
            for j in range(self._held(b)):
                self.refs[self.table[b][j]] -= 1
        for a, b in pairs:
            whole, part = lens[a] // self.page, lens[a] % self.page
            new = table[a][:whole]
            if part:
                p = next(spare)
                self.contents[p] = contents[table[a][whole]]
                new.append(p)
            for j, p in enumerate(new):
                self.refs[p] = 1 if part and j == whole else self.refs[p] + 1
            self.table[b] = new + [-1] * (len(table[a]) - len(new))
            self.lens[b] = lens[a]

    def compact(self):
        L = sum(r > 0 for r in self.refs)
        frm = [p for p in range(L, len(self.refs)) if self.refs[p] > 0]
        to = [p for p in range(L) if self.refs[p] == 0]
        place = dict(zip(frm, to))
        for a, b in place.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.contents[b] = self.contents[a]
        self.table = [[place.get(p, p) for p in row] for row in self.table]
