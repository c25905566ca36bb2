"""The paged key/value cache on the GPU against a 64-bit model: attention of
new tokens over pages, the pages' bookkeeping, and both together."""

import math
import random

import pytest
import torch

import paged_testutil as pt

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
OK, ERR_INDEX, ERR_PAGES = 0, 7, 8            # lizard_status
IMPL_AUTO, IMPL_SIMT = 0, 1


def workspace_status(ws, stream=None):
    from gated_linear_sliding_chunkwise_b200 import lizard
    return lizard.workspace_status(ws, stream)


@pytest.fixture(scope="module")
def paged():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gated_linear_sliding_chunkwise_b200 import paged
    return paged


def _batch(seqs, *, H, Hkv, d, dtype, gap=2, seed=1):
    """q, k, v and cu_q for (new tokens, length) pairs; `gap` rows of q follow the last sequence."""
    gen = torch.Generator().manual_seed(seed)
    cu = [0]
    for n, _ in seqs:
        cu.append(cu[-1] + n)
    T = cu[-1] + gap
    q = torch.randn(T, H, d, generator=gen).to(dtype)
    k = torch.randn(T, Hkv, d, generator=gen).to(dtype)
    v = torch.randn(T, Hkv, d, generator=gen).to(dtype)
    return q, k, v, torch.tensor(cu, dtype=torch.int32)


def _append(c, k, v, cu, layer=0, row=None):
    """The new tokens into the model's pages."""
    page = c["k_pages"].shape[3]
    for b in range(len(cu) - 1):
        r = b if row is None else int(row[b])
        n, s = int(cu[b + 1] - cu[b]), int(c["lens"][r])
        for i in range(n):
            p = s - n + i
            if p >= 0:
                pid = int(c["table"][r, p // page])
                c["k_pages"][layer, pid, :, p % page] = k[int(cu[b]) + i]
                c["v_pages"][layer, pid, :, p % page] = v[int(cu[b]) + i]


def _cuda(c):
    return {n: t.cuda() for n, t in c.items()}


def _run(paged, seqs, *, H, Hkv, d, page, dtype, window=0, sinks=0, impl=IMPL_AUTO, give=True, fill=0.0, gap=2,
         layers=1, layer=0, scale=0.0, row=None, seed=0, edit=None, max_pages=None):
    """One call against the model; returns what a test may look at further."""
    lens = [s for _, s in seqs]
    if row is not None:                       # sequence b on table row row[b]
        by_row = [0] * (max(row) + 1)
        for b, r in enumerate(row):
            by_row[r] = lens[b]
        lens = by_row
    c = pt.build(lens, Hkv=Hkv, d=d, page=page, dtype=dtype, layers=layers, seed=seed, fill=fill,
                 max_pages=max_pages)
    q, k, v, cu = _batch(seqs, H=H, Hkv=Hkv, d=d, dtype=dtype, gap=gap, seed=seed + 1)
    if edit:
        edit(c, q, k, v)
    g = _cuda(c)
    out = torch.full_like(q, 7.0).cuda()
    rt = None if row is None else torch.tensor(row, dtype=torch.int32).cuda()
    r = paged.attn(q.cuda(), k.cuda() if give else None, v.cuda() if give else None, g["k_pages"], g["v_pages"],
                   g["table"], g["lens"], cu.cuda(), max_q=max([n for n, _ in seqs] + [1]), row=rt, layer=layer,
                   window=window, sinks=sinks, softmax_scale=scale, want_lse=True, impl=impl, out=out)
    torch.cuda.synchronize()
    assert workspace_status(r["workspace"]) == OK
    if give:
        _append(c, k, v, cu, layer, row)
    for name in ("k_pages", "v_pages"):       # pages hold exactly what the model's hold
        same = (g[name].cpu() == c[name]) | (torch.isnan(g[name].cpu()) & torch.isnan(c[name]))
        assert same.all(), name
    want = pt.attention(q, c["k_pages"][layer], c["v_pages"][layer], c["table"], c["lens"], cu, window=window,
                        sinks=sinks, scale=scale or None, row=row)
    pt.check_attention(f"{seqs[:3]} H{H}/{Hkv} d{d} p{page}", r["o"], r["lse"], want, d, dtype,
                       rounded_weights=dtype == BF16 and impl != IMPL_SIMT)
    end = int(cu[-1])
    assert (r["o"][end:] == 7.0).all(), "rows behind the last sequence"
    return r, c, g


# ---------------------------------------------------------------- attention
IMPLS = [(FP32, IMPL_AUTO), (FP32, IMPL_SIMT), (BF16, IMPL_SIMT), (BF16, IMPL_AUTO)]
IDS = ["fp32", "fp32-simt", "bf16-simt", "bf16"]


@pytest.mark.parametrize("dtype,impl", IMPLS, ids=IDS)
@pytest.mark.parametrize("H,Hkv,d,page", [(8, 2, 128, 64), (4, 4, 64, 16), (7, 1, 64, 32), (5, 1, 128, 128),
                                          (64, 1, 64, 64)])
def test_single_tokens(paged, dtype, impl, H, Hkv, d, page):
    """Decoding: lengths of one token, around a page and a tile, several tiles."""
    seqs = [(1, s) for s in (1, 2, page - 1, page, page + 1, 63, 64, 65, 127, 128, 129, 300)]
    _run(paged, seqs, H=H, Hkv=Hkv, d=d, page=page, dtype=dtype, impl=impl)


@pytest.mark.parametrize("dtype,impl", IMPLS, ids=IDS)
@pytest.mark.parametrize("H,Hkv,d,page,window,sinks", [
    (8, 2, 128, 64, 0, 0), (4, 4, 64, 16, 50, 3), (6, 2, 64, 128, 1, 0), (7, 1, 128, 32, 129, 200), (3, 3, 64, 16, 64, 64),
    (24, 1, 64, 16, 40, 0)])
def test_chunks(paged, dtype, impl, H, Hkv, d, page, window, sinks):
    """Ragged chunks: whole prompts, ends of long ones, nothing at all."""
    seqs = [(5, 5), (0, 40), (77, 77), (1, 200), (0, 0), (3, 131), (130, 261), (2, 2), (64, 64)]
    _run(paged, seqs, H=H, Hkv=Hkv, d=d, page=page, dtype=dtype, impl=impl, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype,impl", IMPLS, ids=IDS)
def test_one_long_sequence_is_split(paged, dtype, impl):
    """A few rows over thousands of keys, so that many CTAs share an item."""
    _run(paged, [(1, 4099)], H=4, Hkv=1, d=128, page=64, dtype=dtype, impl=impl)
    _run(paged, [(9, 2500), (1, 3)], H=8, Hkv=2, d=64, page=16, dtype=dtype, impl=impl)
    _run(paged, [(40, 1700), (1, 900)], H=8, Hkv=2, d=64, page=16, dtype=dtype, impl=impl, window=700, sinks=130)


@pytest.mark.parametrize("dtype,impl", IMPLS, ids=IDS)
def test_rows_without_keys(paged, dtype, impl):
    """Fewer tokens in the cache than new ones: the first rows stand before the
    sequence and see nothing (zeros, -inf); none of them is written to a page."""
    _run(paged, [(6, 4), (3, 0), (20, 19), (40, 7)], H=4, Hkv=2, d=64, page=16, dtype=dtype, impl=impl)


@pytest.mark.parametrize("dtype,impl", IMPLS, ids=IDS)
@pytest.mark.parametrize("fill", [math.nan, math.inf])
def test_contents_of_unused_slots_do_not_matter(paged, dtype, impl, fill):
    """Slots behind a sequence's last token and pages of nobody hold NaN or infinity."""
    for give in (True, False):
        _run(paged, [(1, 70), (40, 45), (17, 130), (1, 16), (200, 333)], H=4, Hkv=2, d=64, page=32, dtype=dtype,
             impl=impl, fill=fill, give=give)
        _run(paged, [(1, 70), (40, 45), (17, 130)], H=8, Hkv=2, d=128, page=128, dtype=dtype, impl=impl, fill=fill,
             give=give, window=33, sinks=2)


@pytest.mark.parametrize("dtype,impl", IMPLS, ids=IDS)
def test_values_that_a_row_does_not_see_do_not_matter(paged, dtype, impl):
    """NaN and infinities in keys and values outside a row's window: rows that do
    not see them are exact, though others of the same tile are not finite."""
    seqs, window = [(60, 200), (1, 150), (3, 150)], 20

    def edit(c, q, k, v):
        page = c["k_pages"].shape[3]
        # 155: seen by some of the rows; 127: the last key before the window of position 147
        for b, j in ((0, 30), (0, 155), (1, 60), (2, 127)):
            p, o = int(c["table"][b, j // page]), j % page
            c["v_pages"][0, p, :, o, 3] = math.nan
            c["v_pages"][0, p, :, o, 5] = math.inf
            if j != 155:
                c["k_pages"][0, p, :, o] = math.nan

    lens = [s for _, s in seqs]
    c = pt.build(lens, Hkv=2, d=64, page=16, dtype=dtype)
    q, k, v, cu = _batch(seqs, H=4, Hkv=2, d=64, dtype=dtype, gap=0)
    edit(c, q, k, v)
    g = _cuda(c)
    r = paged.attn(q.cuda(), None, None, g["k_pages"], g["v_pages"], g["table"], g["lens"], cu.cuda(), max_q=60,
                   window=window, want_lse=True, impl=impl)
    o = r["o"].cpu()
    pos = torch.arange(60) + 140
    hit = (pos >= 155) & (pos < 155 + window)
    assert torch.isnan(o[:60][hit][:, :, 3]).all()
    assert not torch.isfinite(o[:60][hit][:, :, 5]).any()
    clean = [i for i in range(64) if i not in (3, 5)]
    assert torch.isfinite(o[:60][~hit]).all() and torch.isfinite(o[60:]).all()
    assert torch.isfinite(o[:60][hit][:, :, clean]).all()
    # against the model with the odd values taken out of it
    for name in ("k_pages", "v_pages"):
        c[name] = torch.nan_to_num(c[name], nan=0.0, posinf=0.0)
    want = list(pt.attention(q, c["k_pages"][0], c["v_pages"][0], c["table"], c["lens"], cu, window=window))
    keep = torch.ones(64, dtype=torch.bool)
    keep[:60] = ~hit
    o[~keep] = 0
    want[0][~keep] = 0
    pt.check_attention("unseen", o, r["lse"], want, 64, dtype, rounded_weights=dtype == BF16 and impl != IMPL_SIMT)


@pytest.mark.parametrize("dtype,impl", IMPLS, ids=IDS)
def test_rows_layers_and_scale(paged, dtype, impl):
    """Table rows in another order than the batch, one layer of several, a scale of the caller's."""
    _run(paged, [(3, 40), (1, 90), (33, 64)], H=4, Hkv=2, d=64, page=16, dtype=dtype, impl=impl, layers=3, layer=2,
         scale=0.31, row=[4, 0, 2])


@pytest.mark.parametrize("dtype,impl", IMPLS, ids=IDS)
def test_large_logits(paged, dtype, impl):
    """Logits of several hundred, rising along the sequence: the running maximum moves at every tile."""
    def edit(c, q, k, v):
        page = c["k_pages"].shape[3]
        q.fill_(4.0)
        for b in range(c["table"].shape[0]):
            for j in range(int(c["lens"][b])):
                c["k_pages"][0, int(c["table"][b, j // page]), :, j % page] = (j % 997) / 64
    _run(paged, [(1, 700), (30, 500)], H=8, Hkv=2, d=64, page=64, dtype=dtype, impl=impl, give=False, edit=edit)


def test_a_wide_table_and_a_batch_of_many(paged):
    """More sequences than a block has threads; a table far wider than any row."""
    gen = random.Random(3)
    seqs = [(gen.choice([0, 1, 1, 2]), gen.randint(2, 40)) for _ in range(1100)]
    _run(paged, seqs, H=2, Hkv=1, d=64, page=16, dtype=BF16, max_pages=4000)


def test_wrong_offsets_rows_lengths_and_pages_are_reported(paged):
    """What the device finds is recorded, the other sequences are computed, nothing else is written."""
    def call(change, dtype=BF16):
        c = pt.build([40, 33, 70], Hkv=2, d=64, page=16, dtype=dtype)
        q, k, v, cu = _batch([(2, 40), (33, 33), (1, 70)], H=4, Hkv=2, d=64, dtype=dtype)
        row = torch.tensor([0, 1, 2], dtype=torch.int32)
        change(c, cu, row)
        g = _cuda(c)
        out = torch.full_like(q, 7.0).cuda()
        r = paged.attn(q.cuda(), k.cuda(), v.cuda(), g["k_pages"], g["v_pages"], g["table"], g["lens"], cu.cuda(),
                       max_q=33, row=row.cuda(), out=out)
        first = workspace_status(r["workspace"])
        assert workspace_status(r["workspace"]) == OK         # reading clears it
        return first, r["o"].cpu(), q, k, v, c, cu

    def table(b, j, p):
        return lambda c, cu, row: c["table"].__setitem__((b, j), p)

    for dtype in (BF16, FP32):
        for change in (table(0, 1, 10 ** 6), table(1, 2, -1), table(2, 0, -2 ** 31),
                       lambda c, cu, row: row.__setitem__(1, 3), lambda c, cu, row: row.__setitem__(0, -1),
                       lambda c, cu, row: c["lens"].__setitem__(2, 10 ** 6),
                       lambda c, cu, row: c["lens"].__setitem__(2, -4),
                       lambda c, cu, row: cu.__setitem__(3, 1000), lambda c, cu, row: cu.__setitem__(0, -1)):
            assert call(change, dtype)[0] == ERR_INDEX
    st, o, q, k, v, c, cu = call(lambda c, cu, row: row.__setitem__(1, 3))
    assert st == ERR_INDEX and (o[2:35] == 7.0).all()          # the one left out
    _append(c, k, v, torch.tensor([0, 2], dtype=torch.int32))
    want = pt.attention(q[:2], c["k_pages"][0], c["v_pages"][0], c["table"], c["lens"], cu[:2])
    pt.check_attention("beside a wrong one", o[:2], None, want, 64, BF16, True)


def test_wrong_rows_and_pages_when_decoding_are_reported(paged):
    """The same for a call of single tokens, which no preparing kernel looks over."""
    def call(change):
        c = pt.build([40, 33, 300], Hkv=2, d=128, page=16, dtype=BF16)
        q, k, v, cu = _batch([(1, 40), (1, 33), (2, 300)], H=4, Hkv=2, d=128, dtype=BF16)
        row = torch.tensor([0, 1, 2], dtype=torch.int32)
        change(c, cu, row)
        g = _cuda(c)
        out = torch.full_like(q, 7.0).cuda()
        ws = torch.full((1 << 23,), 255, dtype=torch.uint8, device="cuda")      # whatever it held before
        paged.attn(q.cuda(), k.cuda(), v.cuda(), g["k_pages"], g["v_pages"], g["table"], g["lens"], cu.cuda(), max_q=2,
                   row=row.cuda(), out=out, workspace=ws)
        return workspace_status(ws), out.cpu(), q, k, v, c

    for change in (lambda c, cu, row: c["table"].__setitem__((2, 5), 10 ** 6),
                   lambda c, cu, row: c["table"].__setitem__((2, 18), -1),      # where the new tokens go
                   lambda c, cu, row: row.__setitem__(0, -3), lambda c, cu, row: c["lens"].__setitem__(0, 10 ** 6),
                   lambda c, cu, row: cu.__setitem__(3, 99)):
        assert call(change)[0] == ERR_INDEX
    assert call(lambda c, cu, row: None)[0] == OK
    st, o, q, k, v, c = call(lambda c, cu, row: row.__setitem__(1, 3))
    assert st == ERR_INDEX and (o[1] == 7.0).all()
    _append(c, k, v, torch.tensor([0, 1], dtype=torch.int32))
    want = pt.attention(q[:1], c["k_pages"][0], c["v_pages"][0], c["table"], c["lens"], torch.tensor([0, 1]))
    pt.check_attention("beside a wrong one", o[:1], None, want, 128, BF16, True)


@pytest.mark.parametrize("dtype,n", [(BF16, 1), (BF16, 40), (FP32, 3)], ids=["bf16-one", "bf16-chunk", "fp32"])
def test_pools_beyond_32_bit_offsets(paged, dtype, n):
    """Pages whose first element lies beyond 2^31 elements, in the second of two layers."""
    Hkv, page, d = 8, 128, 128
    per = Hkv * page * d
    P = (1 << 31) // per // 2 + 40
    kp = torch.empty(2, P, Hkv, page, d, dtype=dtype, device="cuda")
    vp = torch.empty_like(kp)
    assert P * per + (P - 5) * per > 1 << 31
    ids = [P - 1, P - 4, P - 2]
    gen = torch.Generator().manual_seed(4)
    for pool in (kp, vp):
        for p in ids:
            pool[1, p] = torch.randn(Hkv, page, d, generator=gen).to(dtype).cuda()
    table, lens = torch.tensor([ids], dtype=torch.int32), torch.tensor([300], dtype=torch.int32)
    q, k, v, cu = _batch([(n, 300)], H=8, Hkv=Hkv, d=d, dtype=dtype, gap=0)
    r = paged.attn(q.cuda(), k.cuda(), v.cuda(), kp, vp, table.cuda(), lens.cuda(), cu.cuda(), max_q=n, layer=1,
                   want_lse=True)
    assert workspace_status(r["workspace"]) == OK
    small = [torch.stack([pool[1, p].cpu() for p in ids]) for pool in (kp, vp)]
    assert torch.equal(small[0][2, :, 300 - 256 - n:300 - 256], k.transpose(0, 1))
    want = pt.attention(q, *small, torch.arange(3, dtype=torch.int32)[None], lens, cu)
    pt.check_attention("far pages", r["o"], r["lse"], want, d, dtype, dtype == BF16)


def test_a_stream_of_the_callers(paged):
    """The calls run on the stream they are given, in its order."""
    c = pt.build([40, 70], Hkv=2, d=64, page=16, dtype=BF16)
    q, k, v, cu = _batch([(1, 40), (20, 70)], H=4, Hkv=2, d=64, dtype=BF16)
    g = _cuda(c)
    dq, dk, dv, dcu = (x.cuda() for x in (q, k, v, cu))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for stream in (s, s.cuda_stream):
        r = paged.attn(dq, dk, dv, g["k_pages"], g["v_pages"], g["table"], g["lens"], dcu, max_q=20, stream=stream)
        outs.append(r["o"])
        ws = paged.free(g["refs"], g["table"], g["lens"], torch.zeros(0, dtype=torch.int32, device="cuda"), page=16,
                        stream=stream)
        assert workspace_status(ws, stream=s) == OK
    s.synchronize()
    _append(c, k, v, cu)
    want = pt.attention(q, c["k_pages"][0], c["v_pages"][0], c["table"], c["lens"], cu)
    for o in outs:
        pt.check_attention("on a stream", o, None, want, 64, BF16, True)


def test_more_new_tokens_than_announced_are_reported(paged):
    c = _cuda(pt.build([40, 40], Hkv=1, d=64, page=16, dtype=BF16))
    q, k, v, cu = _batch([(2, 40), (3, 40)], H=1, Hkv=1, d=64, dtype=BF16)
    r = paged.attn(q.cuda(), k.cuda(), v.cuda(), c["k_pages"], c["v_pages"], c["table"], c["lens"], cu.cuda(), max_q=2)
    assert workspace_status(r["workspace"]) == ERR_INDEX


def test_no_tokens(paged):
    c = _cuda(pt.build([4], Hkv=1, d=64, page=16, dtype=BF16))
    q = torch.zeros(0, 1, 64, dtype=BF16, device="cuda")
    r = paged.attn(q, None, None, c["k_pages"], c["v_pages"], c["table"], c["lens"],
                   torch.zeros(2, dtype=torch.int32, device="cuda"), max_q=0)
    assert r["o"].shape == (0, 1, 64) and workspace_status(r["workspace"]) == OK


@pytest.mark.parametrize("dtype,impl", IMPLS, ids=IDS)
def test_same_call_same_bits(paged, dtype, impl):
    """No result depends on the order in which CTAs finish."""
    seqs = [(1, 3000), (100, 900), (7, 7), (1, 1)]
    c = _cuda(pt.build([s for _, s in seqs], Hkv=2, d=128, page=64, dtype=dtype))
    q, k, v, cu = (x.cuda() for x in _batch(seqs, H=8, Hkv=2, d=128, dtype=dtype, gap=0))
    first = None
    for _ in range(5):
        r = paged.attn(q, k, v, c["k_pages"], c["v_pages"], c["table"], c["lens"], cu, max_q=100, want_lse=True,
                       impl=impl)
        if first is None:
            first = r
        assert torch.equal(r["o"], first["o"]) and torch.equal(r["lse"], first["lse"])


# -------------------------------------------------------------- bookkeeping
def _same(m, c):
    assert c["refs"].tolist() == m.refs
    assert c["table"].tolist() == m.table
    assert c["lens"].tolist() == m.lens


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("page,P,rows,seed", [(16, 300, 24, 0), (128, 40, 5, 1), (32, 5000, 60, 2), (64, 20000, 700, 3)])
def test_random_bookkeeping_follows_the_model(paged, page, P, rows, seed):
    """A long run of reserve, free, fork and compact calls: every count, entry
    and length after each, and the pages' contents at the end."""
    gen = random.Random(seed)
    MP = 12
    layers, Hkv, d = 2, 1, 64
    ids = torch.arange(P, dtype=torch.float32).reshape(1, P, 1, 1, 1) + torch.tensor([0.25, 0.5]).reshape(2, 1, 1, 1, 1)
    kp = ids.expand(layers, P, Hkv, page, d).contiguous().cuda()
    vp = (-kp).contiguous()
    c = dict(refs=torch.zeros(P, dtype=torch.int32), table=torch.full((rows, MP), -1, dtype=torch.int32),
             lens=torch.zeros(rows, dtype=torch.int32))
    m = pt.Model(c["refs"], c["table"], c["lens"], page)
    c = _cuda(c)
    for step in range(40):
        op = gen.choice(["reserve", "reserve", "fork", "fork", "free", "compact"])
        some = gen.sample(range(rows), gen.randint(1, rows))
        if op == "reserve":
            room = sum(r == 0 for r in m.refs)
            grow = []
            for r in some:
                most = min(MP * page - m.lens[r], gen.choice([0, 1, page, 3 * page]))
                g = gen.randint(0, max(0, most))
                need = pt.ceil_div(m.lens[r] + g, page) - m._held(r)
                if need > room:
                    g = need = 0
                room -= need
                grow.append(g)
            m.reserve(some, grow)
            ws = paged.reserve(c["refs"], c["table"], c["lens"], _ints(some), _ints(grow), page=page)
        elif op == "free":
            some = some[: max(1, rows // 3)]
            m.free(some)
            ws = paged.free(c["refs"], c["table"], c["lens"], _ints(some), page=page)
        elif op == "fork":
            src = [gen.randrange(rows) for _ in some]
            if sum(m.lens[a] % page != 0 and a != b for a, b in zip(src, some)) > sum(r == 0 for r in m.refs):
                continue
            m.fork(src, some)
            ws = paged.fork(kp, vp, c["refs"], c["table"], c["lens"], _ints(src), _ints(some))
        else:
            m.compact()
            if step % 2:
                c["table"], c["refs"] = paged.compact(kp, vp, c["refs"], c["table"])
                ws = None
            else:
                ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
                paged.compact(kp, vp, c["refs"], c["table"], table_out=c["table"], refs_out=c["refs"], workspace=ws)
        assert ws is None or workspace_status(ws) == OK
        _same(m, c)
    got = kp[:, :, 0, 0, 0].cpu()
    live = torch.tensor([r > 0 for r in m.refs])
    want = torch.tensor(m.contents, dtype=torch.float32)
    assert torch.equal(got[0][live], want[live] + 0.25) and torch.equal(got[1][live], want[live] + 0.5)
    assert torch.equal(kp, kp[:, :, :1, :1, :1].expand_as(kp)) and torch.equal(vp, -kp)   # whole pages


def _small(page=16, P=10, rows=4, MP=3):
    return dict(refs=torch.zeros(P, dtype=torch.int32).cuda(), lens=torch.zeros(rows, dtype=torch.int32).cuda(),
                table=torch.full((rows, MP), -1, dtype=torch.int32).cuda(), page=page,
                k=torch.zeros(1, P, 1, page, 64, device="cuda"), v=torch.zeros(1, P, 1, page, 64, device="cuda"))


def test_what_is_not_allowed_changes_nothing(paged):
    """Too few pages, rows out of range or listed twice, lengths past the table,
    broken tables: a status, and every array as it was."""
    s = _small()
    args = (s["refs"], s["table"], s["lens"])
    assert workspace_status(paged.reserve(*args, _ints([1, 3]), _ints([40, 17]), page=16)) == OK

    def unchanged(want, call, prepare=None):
        if prepare:
            prepare()
        before = [x.clone() for x in (*args, s["k"], s["v"])]
        assert workspace_status(call()) == want
        for x, y in zip(before, (*args, s["k"], s["v"])):
            assert torch.equal(x, y)

    def reserve(rows, grow):
        return lambda: paged.reserve(*args, _ints(rows), _ints(grow), page=16)

    unchanged(ERR_INDEX, reserve([1, 1], [1, 1]))
    unchanged(ERR_INDEX, reserve([0, 4], [1, 1]))
    unchanged(ERR_INDEX, reserve([-1], [1]))
    unchanged(ERR_INDEX, reserve([0], [49]))                       # three pages of 16
    unchanged(ERR_INDEX, reserve([0], [-1]))
    unchanged(ERR_INDEX, reserve([1], [2 ** 31 - 1]))
    unchanged(ERR_PAGES, reserve([0, 2], [48, 48]))                # 6 pages, 5 are free
    unchanged(ERR_INDEX, lambda: paged.free(*args, _ints([1, 1]), page=16))
    unchanged(ERR_INDEX, lambda: paged.free(*args, _ints([9]), page=16))

    def fork(src, rows):
        return lambda: paged.fork(s["k"], s["v"], *args, _ints(src), _ints(rows))

    unchanged(ERR_INDEX, fork([1, 1], [0, 0]))
    unchanged(ERR_INDEX, fork([7], [0]))
    unchanged(ERR_INDEX, fork([1], [-7]))
    assert workspace_status(paged.reserve(*args, _ints([0, 2]), _ints([32, 48]), page=16)) == OK   # all pages held
    unchanged(ERR_PAGES, fork([1], [0]))
    unchanged(OK, fork([1, 3], [1, 3]))                            # each row continues from itself
    s["table"][1, 0] = 99
    unchanged(ERR_INDEX, lambda: paged.free(*args, _ints([1]), page=16))
    unchanged(ERR_INDEX, fork([1], [0]))
    unchanged(ERR_INDEX, fork([0], [1]))
    # compact leaves such an entry alone and says so
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    t, r = paged.compact(s["k"], s["v"], s["refs"], s["table"], workspace=ws)
    assert workspace_status(ws) == ERR_INDEX and int(t[1, 0]) == 99


def test_beams_trade_places(paged):
    """One call that lets rows continue from one another in a circle."""
    s = _small(P=12)
    args = (s["refs"], s["table"], s["lens"])
    m = pt.Model(*(x.cpu() for x in args), 16)
    m.reserve([0, 1, 2], [20, 33, 16])
    paged.reserve(*args, _ints([0, 1, 2]), _ints([20, 33, 16]), page=16)
    for _ in range(4):
        m.fork([1, 2, 0, 1], [0, 1, 2, 3])
        assert workspace_status(paged.fork(s["k"], s["v"], *args, _ints([1, 2, 0, 1]), _ints([0, 1, 2, 3]))) == OK
        _same(m, s)


@pytest.mark.parametrize("layers", [1, 8])
def test_branches_of_one_source_copy_its_last_page(paged, layers):
    """Few and many bytes (the latter share their loads): runs of one source,
    the same source again later, a source without a part-filled page."""
    page, Hkv, d, P, MP = 128, 8, 128, 24, 3
    gen = torch.Generator(device="cuda").manual_seed(layers)
    kp = torch.randn(layers, P, Hkv, page, d, generator=gen, device="cuda")
    vp = torch.randn(layers, P, Hkv, page, d, generator=gen, device="cuda")
    s = dict(refs=torch.zeros(P, dtype=torch.int32).cuda(), lens=torch.zeros(13, dtype=torch.int32).cuda(),
             table=torch.full((13, MP), -1, dtype=torch.int32).cuda())
    args = (s["refs"], s["table"], s["lens"])
    m = pt.Model(*(x.cpu() for x in args), page)
    m.reserve([0, 1, 2, 3], [5, 300, 256, 130])
    paged.reserve(*args, _ints([0, 1, 2, 3]), _ints([5, 300, 256, 130]), page=page)
    before = kp.clone(), vp.clone()
    src, row = [0, 0, 1, 0, 2, 0, 3, 3, 1], [4, 5, 6, 7, 8, 9, 10, 11, 12]
    m.fork(src, row)
    assert workspace_status(paged.fork(kp, vp, *args, _ints(src), _ints(row))) == OK
    _same(m, s)
    where = torch.tensor(m.contents).cuda()
    assert torch.equal(kp, before[0][:, where]) and torch.equal(vp, before[1][:, where])


def test_empty_lists_and_pools(paged):
    s = _small()
    args = (s["refs"], s["table"], s["lens"])
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert workspace_status(paged.reserve(*args, none, none, page=16)) == OK
    assert workspace_status(paged.free(*args, none, page=16)) == OK
    t, r = paged.compact(s["k"], s["v"], s["refs"], s["table"])      # nothing is live
    assert torch.equal(t, s["table"]) and torch.equal(r, s["refs"])
    s["refs"].fill_(1)                                                # everything is
    t, r = paged.compact(s["k"], s["v"], s["refs"], s["table"])
    assert torch.equal(r, s["refs"])


# ------------------------------------------------------------ used together
def _serve(paged, dtype, steps, graph):
    """Prompts in chunks, forks, decoding, leaving, closing up: outputs of every call."""
    H, Hkv, d, page, rows, MP, P, layers = 4, 2, 64, 16, 6, 8, 40, 2
    gen = torch.Generator().manual_seed(5)
    kp = torch.full((layers, P, Hkv, page, d), math.nan).to(dtype)
    c = _cuda(dict(k_pages=kp, v_pages=kp.clone(), refs=torch.zeros(P, dtype=torch.int32),
                   table=torch.full((rows, MP), -1, dtype=torch.int32), lens=torch.zeros(rows, dtype=torch.int32)))
    book = (c["refs"], c["table"], c["lens"])
    history = [[[] for _ in range(layers)] for _ in range(rows)]      # the tokens' (k, v) of each row

    def attend(row, n):
        for layer in range(layers):
            T = sum(n)
            q, k, v = (torch.randn(T, h, d, generator=gen).to(dtype) for h in (H, Hkv, Hkv))
            cu = torch.tensor([0] + list(torch.tensor(n).cumsum(0)), dtype=torch.int32)
            r = paged.attn(q.cuda(), k.cuda(), v.cuda(), c["k_pages"], c["v_pages"], c["table"], c["lens"], cu.cuda(),
                           max_q=max(n), row=_ints(row), layer=layer, window=40, sinks=2, want_lse=True)
            assert workspace_status(r["workspace"]) == OK
            for b, x in enumerate(row):
                for i in range(int(cu[b]), int(cu[b + 1])):
                    history[x][layer].append((k[i], v[i]))
                # the model: this row's history as one contiguous cache
                hist = history[x][layer]
                kk, vv = (torch.stack([e[j] for e in hist]) for j in (0, 1))
                pad = pt.ceil_div(len(hist), page) * page - len(hist)
                pages = [torch.nn.functional.pad(y, (0, 0, 0, 0, 0, pad)).reshape(-1, page, Hkv, d).transpose(1, 2)
                         for y in (kk, vv)]
                want = pt.attention(q[int(cu[b]):int(cu[b + 1])], *pages, torch.arange(pages[0].shape[0])[None],
                                    torch.tensor([len(hist)]), torch.tensor([0, n[b]]), window=40, sinks=2)
                pt.check_attention(f"row {x} layer {layer}", r["o"][int(cu[b]):int(cu[b + 1])],
                                   r["lse"][int(cu[b]):int(cu[b + 1])], want, d, dtype, dtype == BF16)

    def reserve(row, n):
        assert workspace_status(paged.reserve(*book, _ints(row), _ints(n), page=page)) == OK

    reserve([0, 1], [37, 50])
    attend([0, 1], [37, 50])
    assert workspace_status(paged.fork(c["k_pages"], c["v_pages"], *book, _ints([0, 0, 1]), _ints([2, 3, 4]))) == OK
    for a, b in ((0, 2), (0, 3), (1, 4)):
        history[b] = [list(x) for x in history[a]]
    for _ in range(steps):
        reserve([0, 2, 3, 4], [1, 1, 2, 1])
        attend([0, 2, 3, 4], [1, 1, 2, 1])
    assert workspace_status(paged.free(*book, _ints([0, 1]), page=page)) == OK
    history[0] = [[] for _ in range(layers)]
    history[1] = [[] for _ in range(layers)]
    paged.compact(c["k_pages"], c["v_pages"], c["refs"], c["table"], table_out=c["table"], refs_out=c["refs"])
    live = int((c["refs"] > 0).sum())
    assert (c["refs"][:live] > 0).all() and (c["refs"][live:] == 0).all()
    reserve([1, 2, 3, 4], [23, 1, 1, 3])
    attend([1, 2, 3, 4], [23, 1, 1, 3])


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_a_serving_run(paged, dtype):
    _serve(paged, dtype, steps=3, graph=False)


def test_a_captured_step_follows_the_lengths(paged):
    """One decoding step (reserve, attention of two layers, with their
    workspaces) captured once and replayed: each replay works on the lengths
    that the one before left.  A second graph with workspaces of its own
    replays on another stream at the same time."""
    H, Hkv, d, page, rows, MP, P, layers = 4, 2, 128, 16, 3, 8, 30, 2

    def world(seed):
        gen = torch.Generator().manual_seed(seed)
        c = _cuda(dict(k_pages=torch.zeros(layers, P, Hkv, page, d).to(BF16),
                       v_pages=torch.zeros(layers, P, Hkv, page, d).to(BF16),
                       refs=torch.zeros(P, dtype=torch.int32), table=torch.full((rows, MP), -1, dtype=torch.int32),
                       lens=torch.zeros(rows, dtype=torch.int32)))
        x = [[torch.randn(20, rows, h, d, generator=gen).to(BF16).cuda() for h in (H, Hkv, Hkv)] for _ in range(layers)]
        return c, x, [[torch.zeros(rows, h, d, dtype=BF16, device="cuda") for h in (H, Hkv, Hkv)] for _ in range(layers)]

    def step(c, tok, out, ws):
        ws[0] = paged.reserve(c["refs"], c["table"], c["lens"], _ints_row, _ones, page=page, workspace=ws[0])
        for layer in range(layers):
            r = paged.attn(*tok[layer], c["k_pages"], c["v_pages"], c["table"], c["lens"], _cu, max_q=1, layer=layer,
                           out=out[layer], workspace=ws[1 + layer])
            ws[1 + layer] = r["workspace"]

    _ints_row, _ones, _cu = _ints([0, 1, 2]), _ints([1, 1, 1]), _ints([0, 1, 2, 3])
    plain, graphs = [], []
    for seed in (1, 2):
        c, x, tok = world(seed)
        out = [torch.zeros(rows, H, d, dtype=BF16, device="cuda") for _ in range(layers)]
        got, ws = [], [None] * (1 + layers)
        for t in range(20):
            for layer in range(layers):
                for dst, srcs in zip(tok[layer], x[layer]):
                    dst.copy_(srcs[t])
            step(c, tok, out, ws)
            got.append([o.clone() for o in out])
        plain.append(got)
        c, x, tok = world(seed)
        out = [torch.zeros(rows, H, d, dtype=BF16, device="cuda") for _ in range(layers)]
        ws = [torch.empty_like(w) for w in ws]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(c, tok, out, ws)
        graphs.append((g, c, x, tok, out, ws))
    streams = [torch.cuda.Stream() for _ in range(2)]
    seen = [[], []]
    torch.cuda.synchronize()
    for t in range(20):
        for w, (g, c, x, tok, out, ws) in enumerate(graphs):
            with torch.cuda.stream(streams[w]):
                for layer in range(layers):
                    for dst, srcs in zip(tok[layer], x[layer]):
                        dst.copy_(srcs[t])
                g.replay()
                seen[w].append([o.clone() for o in out])
    torch.cuda.synchronize()
    for w in range(2):
        assert graphs[w][1]["lens"].tolist() == [20] * rows
        for a, b in zip(plain[w], seen[w]):
            for y, z in zip(a, b):
                assert torch.equal(y, z)
        for ws in graphs[w][5]:
            assert workspace_status(ws) == OK


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_a_captured_mixed_batch_follows_lengths_and_offsets(paged, dtype):
    """Decoding tokens and a chunk in one captured call (every kernel of the
    attention): replays read the lengths, offsets and tables of the moment."""
    H, Hkv, d, page = 8, 2, 64, 16
    most = 600
    c = pt.build([most] * 3, Hkv=Hkv, d=d, page=page, dtype=dtype)
    q, k, v, cu = _batch([(1, most), (70, most), (2, most)], H=H, Hkv=Hkv, d=d, dtype=dtype, gap=0)
    g = _cuda(c)
    dq, dk, dv, dcu = (x.cuda() for x in (q, k, v, cu))
    out = torch.zeros_like(dq)

    def call(ws=None):
        return paged.attn(dq, dk, dv, g["k_pages"], g["v_pages"], g["table"], g["lens"], dcu, max_q=73, window=200,
                          sinks=5, out=out, workspace=ws)["workspace"]

    ws = torch.empty_like(call())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ws)
    for lens, at in (([600, 600, 600], [0, 1, 71, 73]), ([17, 71, 2], [0, 1, 71, 73]), ([599, 80, 333], [0, 73, 73, 73]),
                     ([300, 1, 64], [0, 0, 1, 73]), ([4, 500, 90], [0, 1, 2, 3])):
        c["lens"] = torch.tensor(lens, dtype=torch.int32)
        cu = torch.tensor(at, dtype=torch.int32)
        c["k_pages"], c["v_pages"] = g["k_pages"].cpu(), g["v_pages"].cpu()
        g["lens"].copy_(c["lens"])
        dcu.copy_(cu)
        out.fill_(7.0)
        for _ in range(2):
            graph.replay()
        assert workspace_status(ws) == OK
        _append(c, k, v, cu)
        want = pt.attention(q, c["k_pages"][0], c["v_pages"][0], c["table"], c["lens"], cu, window=200, sinks=5)
        pt.check_attention(f"replayed {lens} {at}", out, None, want, d, dtype, dtype == BF16)
        assert (out[at[-1]:] == 7.0).all()
