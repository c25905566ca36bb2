"""The paged cache on the GPU where calls meet one another or go wrong late:
refusals found behind the list's checks, memory of other streams, rows that are
computed again, results that must not depend on what ran before."""

import math
import random
import sys
import threading
import time

import pytest
import torch

import paged_testutil as pt
from test_gpu_paged import BF16, ERR_INDEX, ERR_PAGES, FP32, IMPL_SIMT, OK, _batch, _cuda, _ints, paged, workspace_status  # noqa: F401

pytestmark = pytest.mark.gpu


def test_too_few_pages_for_a_long_list_change_nothing(paged):
    """A list that the eight CTAs of a cluster work on, one page short: the
    shortage is found after the list's checks have passed, by one CTA while
    the others may be behind it.  Refused many times, with every array as it
    was; with one page more the same list goes through."""
    page, rows, MP, P = 16, 2000, 3, 6000
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    table = torch.full((rows, MP), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    pool = torch.zeros(1, P, 1, page, 64, device="cuda")
    book = (refs, table, lens)
    some, half = _ints(range(rows)), rows // 2
    refs[2 * rows - 1:] = 1                                  # 2 * rows - 1 pages are free
    grow = torch.full((rows,), 17, dtype=torch.int32, device="cuda")      # two pages each

    def refused(call, times=200):
        before = [x.clone() for x in (*book, pool)]
        for _ in range(times):
            assert workspace_status(call()) == ERR_PAGES
        for x, y in zip(before, (*book, pool)):
            assert torch.equal(x, y)

    refused(lambda: paged.reserve(*book, some, grow, page=page))
    # half of the rows get a part-filled page; then each is to be forked, with one page too few
    refs[:] = 0
    assert workspace_status(paged.reserve(*book, some[:half], torch.ones_like(grow[:half]), page=page)) == OK
    refs[rows - 1:] = 1                                      # half - 1 pages are left
    refused(lambda: paged.fork(pool, pool.clone(), *book, some[:half], some[half:]))
    refs[P - 1] = 0
    assert workspace_status(paged.fork(pool, pool.clone(), *book, some[:half], some[half:])) == OK
    assert (lens == 1).all() and (refs > 0).all()
    assert torch.equal(table[half:, 0].sort().values[:-1], _ints(range(half, rows - 1)))
    assert int(table[half:, 0].max()) == P - 1


def test_compact_says_what_it_found_without_a_workspace_of_the_callers(paged):
    page, P = 16, 8
    pool = torch.zeros(1, P, 1, page, 64, device="cuda")
    refs, table = _ints([0, 0, 1, 0, 1, 0, 0, 1]), _ints([[4, 2, -1], [7, -1, -1]])
    r = paged.compact(pool, pool.clone(), refs, table)
    t, n = r
    assert workspace_status(r.workspace) == OK
    assert t.tolist() == [[0, 2, -1], [1, -1, -1]] and n.tolist() == [1, 1, 1, 0, 0, 0, 0, 0]
    for wrong in (5, 8, 2 ** 31 - 1):          # nobody's page, and none of the pool's
        table[1, 1] = wrong
        r = paged.compact(pool, pool.clone(), refs, table)
        assert workspace_status(r.workspace) == ERR_INDEX
        assert r[0].tolist() == [[0, 2, -1], [1, wrong, -1]]


# ------------------------------------------------------------------ streams
def _calls(paged):
    """Each entry point as a call that takes a stream and gives its tensors."""
    c = _cuda(pt.build([40, 70], Hkv=2, d=64, page=16, dtype=BF16))
    q, k, v, cu = (x.cuda() for x in _batch([(1, 40), (20, 70)], H=4, Hkv=2, d=64, dtype=BF16))
    book, none, one, zero = (c["refs"], c["table"], c["lens"]), _ints([]), _ints([1]), _ints([0])

    def attn(stream):
        r = paged.attn(q, k, v, c["k_pages"], c["v_pages"], c["table"], c["lens"], cu, max_q=20, want_lse=True,
                       stream=stream)
        return [r["o"], r["lse"], r["workspace"]]

    return dict(attn=attn,
                reserve=lambda stream: [paged.reserve(*book, zero, zero, page=16, stream=stream)],
                free=lambda stream: [paged.free(*book, none, page=16, stream=stream)],
                fork=lambda stream: [paged.fork(c["k_pages"], c["v_pages"], *book, one, one, stream=stream)],
                compact=lambda stream: list(paged.compact(c["k_pages"], c["v_pages"], c["refs"], c["table"],
                                                          stream=stream)))


def _spans(tensors):
    return [(t.data_ptr(), t.data_ptr() + t.nbytes) for t in tensors]


def _overlap(x, y):
    return [(a, b) for a in x for b in y if a[0] < b[1] and b[0] < a[1]]


@pytest.mark.parametrize("name", ["attn", "reserve", "free", "fork", "compact"])
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_outputs_and_workspaces_belong_to_the_stream_of_the_call(paged, name, handle):
    """No block of the current stream's memory, where work may still be pending
    on it, is given to a call on another stream, and none of that call's goes
    back to the current stream while the other one runs."""
    call = _calls(paged)[name]
    s = torch.cuda.Stream()
    on = s.cuda_stream if handle else s
    torch.cuda.synchronize()
    sizes = [t.nbytes for t in call(None)]
    torch.cuda.synchronize()

    def blocks():                              # the sizes that the call wants, from the current stream's memory
        return [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]

    freed = _spans(blocks())                   # recycled at once
    out = call(on)
    assert not _overlap(freed, _spans(out))
    gone = _spans(out)
    del out                                    # dropped while the stream may be at work
    assert not _overlap(gone, _spans(blocks()))
    torch.cuda.synchronize()


def test_a_call_on_another_stream_leaves_the_current_stream_alone(paged):
    torch.cuda.synchronize()
    call, s, here = _calls(paged)["attn"], torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    want = call(None)
    torch.cuda.synchronize()
    got = call(s)
    assert torch.cuda.current_stream() == here
    s.synchronize()
    for x, y in zip(want[:2], got[:2]):
        assert torch.equal(x[:21], y[:21])     # the rows of the sequences


def test_other_threads_run_while_a_call_launches(paged):
    """The interpreter's lock is free during the launches.  With a switch
    interval that never ends, another thread only gets its turn where a call
    gives up the lock."""
    turns, stop, ready = [0], threading.Event(), threading.Event()

    def other():
        ready.set()
        while not stop.is_set():
            turns[0] += 1
            time.sleep(0)                      # gives up the lock at once

    calls = _calls(paged)
    for call in calls.values():
        call(None)
    torch.cuda.synchronize()
    before, kept = sys.getswitchinterval(), []
    thread = threading.Thread(target=other)
    try:
        sys.setswitchinterval(1000.0)
        thread.start()
        ready.wait()
        for name in ("attn", "fork"):
            seen = turns[0]
            for _ in range(500):
                kept.append(calls[name](None))
                if turns[0] != seen:
                    break
            assert turns[0] != seen, name
    finally:
        sys.setswitchinterval(before)
        stop.set()
        thread.join()
    torch.cuda.synchronize()


# --------------------------------------------------- rows computed again
def _long_case(seqs, *, H, Hkv, d, page, seed):
    """A cache on the GPU with pages in order, too long for the model's builder."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    used = [pt.ceil_div(s, page) for _, s in seqs]
    P = sum(used)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(BF16)

    table, at = torch.full((len(seqs), max(used)), -1, dtype=torch.int32), 0
    for b, n in enumerate(used):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    T = sum(n for n, _ in seqs)
    cu = torch.tensor([0] + [n for n, _ in seqs]).cumsum(0).to(torch.int32)
    return dict(q=normal(T, H, d), k_pages=normal(1, P, Hkv, page, d), v_pages=normal(1, P, Hkv, page, d),
                table=table.cuda(), lens=_ints([s for _, s in seqs]), cu=cu.cuda())


def _check_tokens(name, c, r, tokens, seqs, d, skip=()):
    """These tokens (sequence, index) against the model; columns `skip` are not finite."""
    keep = [x for x in range(d) if x not in skip]
    cu = c["cu"].tolist()
    for b, i in tokens:
        n, s = seqs[b]
        t, p = cu[b] + i, s - n + i
        ids = c["table"][b, : pt.ceil_div(s, c["k_pages"].shape[3])].long()
        pools = [c[x][0, ids].cpu() for x in ("k_pages", "v_pages")]
        pools[1][..., list(skip)] = 0
        want = pt.attention(c["q"][t:t + 1].cpu(), *pools, torch.arange(len(ids))[None], torch.tensor([p + 1]),
                            torch.tensor([0, 1]))
        got = r["o"][t:t + 1].clone()
        assert not torch.isfinite(got[..., list(skip)]).any()
        got[..., list(skip)] = 0
        assert torch.isfinite(got[..., keep]).all()
        pt.check_attention(f"{name} {b} {i}", got, r["lse"][t:t + 1], want, d, BF16, True)


@pytest.mark.parametrize("H,Hkv,d,page,seqs", [
    (16, 4, 128, 64, [(1500, 16384), (77, 300), (40, 2000)]),              # chunks; one prompt is computed again
    (16, 4, 64, 16, [(1, 16384)] * 6 + [(1, 700), (2, 5000)]),             # decoding
], ids=["chunks", "decoding"])
def test_an_infinite_value_of_a_long_sequence_leaves_the_others_alone(paged, H, Hkv, d, page, seqs):
    """Every row of a long sequence sees an infinite value and is computed
    again, key by key: no wait of the call's kernels gives up meanwhile, and
    the other sequences of the batch are what they are without it."""
    long = [b for b, (_, s) in enumerate(seqs) if s == 16384]
    c = _long_case(seqs, H=H, Hkv=Hkv, d=d, page=page, seed=3)

    def call():
        r = paged.attn(c["q"], None, None, c["k_pages"], c["v_pages"], c["table"], c["lens"], c["cu"],
                       max_q=max(n for n, _ in seqs), want_lse=True)
        assert workspace_status(r["workspace"]) == OK
        return r

    plain = call()
    for b in long:
        c["v_pages"][0, int(c["table"][b, 0]), :, 3, 5] = torch.inf
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    r = call()
    end.record()
    torch.cuda.synchronize()
    print(f"PAGED rows computed again: {start.elapsed_time(end):.1f} ms")
    cu = c["cu"].tolist()
    for b in range(len(seqs)):
        if b not in long:
            assert torch.equal(plain["o"][cu[b]:cu[b + 1]], r["o"][cu[b]:cu[b + 1]])
            assert torch.equal(plain["lse"][cu[b]:cu[b + 1]], r["lse"][cu[b]:cu[b + 1]])
    _check_tokens("again", c, r, [(long[0], 0), (long[-1], seqs[long[-1]][0] - 1)], seqs, d, skip=(5,))
    _check_tokens("beside", c, r, [(len(seqs) - 1, 0)], seqs, d)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_portable_rows_computed_again_keep_the_second_result(paged, dtype):
    """A row is written once with what the tile's products gave and once more
    key by key: what stays is the second, in every column, run after run."""
    seqs, window = [(64, 64)] * 40, 9
    c = pt.build([s for _, s in seqs], Hkv=1, d=64, page=16, dtype=dtype)
    q, k, v, cu = _batch(seqs, H=1, Hkv=1, d=64, dtype=dtype, gap=0)
    clean = {n: c[n].clone() for n in ("k_pages", "v_pages")}
    for b in range(len(seqs)):                 # value 0: seen by tokens 0 .. 8, in the tile of all 64
        c["v_pages"][0, int(c["table"][b, 0]), :, 0] = torch.inf
    g = _cuda(c)
    want = pt.attention(q, clean["k_pages"][0], clean["v_pages"][0], c["table"], c["lens"], cu, window=window)
    sees = torch.arange(64).repeat(len(seqs)) < window
    for _ in range(20):
        r = paged.attn(q.cuda(), None, None, g["k_pages"], g["v_pages"], g["table"], g["lens"], cu.cuda(), max_q=64,
                       window=window, want_lse=True, impl=IMPL_SIMT)
        o = r["o"].cpu()
        assert (o[sees] == torch.inf).all()
        o[sees] = want[0][sees].to(dtype)
        pt.check_attention("portable again", o, r["lse"], want, 64, dtype, rounded_weights=False)


@pytest.mark.parametrize("d", [64, 128])
def test_bits_do_not_depend_on_the_call_before(paged, d):
    """Seven heads to a kv head fill 126 of a tile's 128 rows: what another call
    left in shared memory for the other two has no say in the results."""
    page, many = 64, 48                         # nine tiles of keys to a CTA
    c = _long_case([(36, 4000)] * many, H=7, Hkv=1, d=d, page=page, seed=8)
    full = torch.randn(32 * many, 8, d, device="cuda").to(BF16)

    def call(q, cu, window):
        r = paged.attn(q, None, None, c["k_pages"], c["v_pages"], c["table"], c["lens"], cu, max_q=36, window=window,
                       want_lse=True)
        assert workspace_status(r["workspace"]) == OK
        return r["o"], r["lse"]

    cu8 = _ints(range(0, 32 * many + 1, 32))
    for window in (0, 1500):
        first = None
        for scale in (0.0, 1.0, 30.0, 1000.0):
            call((full * scale).to(BF16), cu8, 0)            # 128 rows in every tile
            got = call(c["q"], c["cu"], window)
            if first is None:
                first = got
            assert torch.equal(first[0], got[0]) and torch.equal(first[1], got[1]), (window, scale)


# Queries of 4 and a key of x in every column have the logit 4 x sqrt(d), in
# log2 units 46.2 x at d = 64 and 65.3 x at d = 128.
@pytest.mark.parametrize("d,x", [(64, 2.25), (64, 3.5), (64, 8.0), (128, 1.625), (128, 2.5)],
                         ids=["104", "162", "369", "106", "163"])
@pytest.mark.parametrize("seqs,H,Hkv,jumps", [
    # a piece of several tiles per CTA, whole items and split ones; keys from the first of the
    # jump on stand out, by up to x, in the middle of the prompt, at a tile's ends, and where
    # only the last of the new tokens see them
    ([(130, 6000)], 8, 8, (300, 2431)), ([(130, 6000)], 8, 8, (2047, 2048)), ([(130, 6000)], 8, 8, (5950, 5999)),
    ([(33, 1500)] * 12, 8, 2, (200, 1490)), ([(33, 1500)] * 24, 7, 1, (129, 1499))])
def test_a_leap_of_the_maximum_within_a_tile(paged, d, x, seqs, H, Hkv, jumps):
    """Logits that rise by more than 2^96, and by more than 2^128, over all
    before them within one tile of keys, in weights formed with the maximum
    from before: such rows are computed again; rows beside them that do not
    see the leap are not touched by it."""
    gen = torch.Generator().manual_seed(11)
    page = 64
    lens = [s for _, s in seqs]
    c = pt.build(lens, Hkv=Hkv, d=d, page=page, dtype=BF16)
    c["k_pages"] /= 64
    q, _, _, cu = _batch(seqs, H=H, Hkv=Hkv, d=d, dtype=BF16, gap=0)
    q.fill_(4.0)
    for b in range(len(seqs)):
        for j in jumps:
            for i, y in enumerate((x, x - 1 / 64)):           # two weights that differ: neither is all of it
                if j + i < lens[b]:
                    c["k_pages"][0, int(c["table"][b, (j + i) // page]), :, (j + i) % page] = y
    g = _cuda(c)
    r = paged.attn(q.cuda(), None, None, g["k_pages"], g["v_pages"], g["table"], g["lens"], cu.cuda(),
                   max_q=max(n for n, _ in seqs), want_lse=True)
    assert workspace_status(r["workspace"]) == OK
    some = [0, len(seqs) - 1] if len(seqs) > 1 else [0]       # the model is slow
    for b in some:
        a, z = int(cu[b]), int(cu[b + 1])
        pick = sorted({*torch.randint(0, z - a, (6,), generator=gen).tolist(), 0, z - a - 1})
        for i in pick:
            p = lens[b] - (z - a) + i
            want = pt.attention(q[a + i:a + i + 1], c["k_pages"][0], c["v_pages"][0], c["table"][b:b + 1],
                                torch.tensor([p + 1]), torch.tensor([0, 1]))
            pt.check_attention(f"leap {b} {i}", r["o"][a + i:a + i + 1], r["lse"][a + i:a + i + 1], want, d, BF16, True)


# --------------------------------------------------------------- precision
@pytest.mark.parametrize("H,Hkv,d,page", [(32, 8, 128, 64), (14, 2, 64, 16), (5, 5, 64, 128)])
def test_decoding_keeps_its_weights_to_16_bits(paged, H, Hkv, d, page):
    """At most 16 rows per key/value head: a weight goes to its product with v
    as two bf16 numbers.  The first is off by half a step, 2^-8 of the weight,
    the second by 2^-8 of that: 2^-16 of it stays, beside the bounds that
    check_attention derives for logits, exp2, sums and the output's rounding."""
    seqs = [(1, 1), (1, 70), (2, 517), (1, 2000), (2, 1300)]
    c = pt.build([s for _, s in seqs], Hkv=Hkv, d=d, page=page, dtype=BF16)
    q, _, _, cu = _batch(seqs, H=H, Hkv=Hkv, d=d, dtype=BF16, gap=0)
    g = _cuda(c)
    r = paged.attn(q.cuda(), None, None, g["k_pages"], g["v_pages"], g["table"], g["lens"], cu.cuda(), max_q=2)
    o, _, A, mag = pt.attention(q, c["k_pages"][0], c["v_pages"][0], c["table"], c["lens"], cu)
    weights = A * (2 * (d + 4) * 2.0 ** -22 * mag + 2.0 ** -20 + 2.0 ** -16).unsqueeze(-1)
    half = torch.finfo(BF16).eps / 2
    err = (r["o"].double().cpu() - o).abs()
    assert (err <= weights * (1 + half) + half * o.abs() + 1e-30).all(), \
        f"worst {float((err / (weights * (1 + half) + half * o.abs() + 1e-30)).max()):.2f} of the bound"


@pytest.mark.parametrize("seqs", [[(1, 70), (2, 1300), (1, 1)], [(90, 400), (1, 33), (300, 300)]], ids=["few", "chunks"])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_the_output_may_be_the_new_keys_or_values(paged, dtype, which, seqs):
    """With as many key/value heads as query heads: the same bits as beside them."""
    c = pt.build([s for _, s in seqs], Hkv=3, d=64, page=16, dtype=dtype)
    q, k, v, cu = (x.cuda() for x in _batch(seqs, H=3, Hkv=3, d=64, dtype=dtype, gap=0))
    outs = []
    for beside in (True, False):
        g = _cuda(c)
        x = dict(k=k.clone(), v=v.clone())
        r = paged.attn(q, x["k"], x["v"], g["k_pages"], g["v_pages"], g["table"], g["lens"], cu,
                       max_q=max(n for n, _ in seqs), out=torch.empty_like(q) if beside else x[which])
        assert workspace_status(r["workspace"]) == OK
        outs.append([r["o"], g["k_pages"], g["v_pages"]])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


# ------------------------------------------- pieces of one and two query tiles
@pytest.mark.parametrize("H,Hkv,d,page,window,sinks", [
    (48, 1, 128, 32, 128, 0), (64, 1, 64, 64, 1, 0), (12, 2, 128, 128, 64, 3), (14, 2, 64, 16, 65, 1),
    (7, 1, 128, 16, 17, 65), (24, 1, 64, 32, 0, 0)])
def test_pieces_with_rows_for_one_query_tile_between_others(paged, H, Hkv, d, page, window, sinks):
    """Hundreds of short sequences, so that a CTA has many pieces in a row: some
    fill one query tile and leave the other's warps nothing, some have rows for
    both, and nearly all end inside a tile of keys."""
    gen = random.Random(H)
    tokens = -(-128 // (H // Hkv))                           # of a query tile, rounded up
    seqs = []
    for _ in range(300):
        n = gen.choice([1, 1, 1, tokens, tokens + 1, 2 * tokens, 4 * tokens]) if gen.random() < 0.5 else 1
        n = min(n, 40)
        seqs.append((n, n + gen.randint(0, 180)))
    c = pt.build([s for _, s in seqs], Hkv=Hkv, d=d, page=page, dtype=BF16)
    q, _, _, cu = _batch(seqs, H=H, Hkv=Hkv, d=d, dtype=BF16, gap=0)
    g = _cuda(c)
    want = [torch.cat(x) for x in zip(*(_plain(q, c, cu, b, s, window, sinks) for b, (_, s) in enumerate(seqs)))]
    for _ in range(10):
        r = paged.attn(q.cuda(), None, None, g["k_pages"], g["v_pages"], g["table"], g["lens"], cu.cuda(), max_q=40,
                       window=window, sinks=sinks, want_lse=True)
        assert workspace_status(r["workspace"]) == OK
        pt.check_attention("pieces", r["o"], r["lse"], want, d, BF16, True)


def _plain(q, c, cu, b, s, window, sinks):
    """The model's attention of one sequence, all its tokens at once."""
    a, z = int(cu[b]), int(cu[b + 1])
    Hkv, page, d = c["k_pages"].shape[2], c["k_pages"].shape[3], q.shape[2]
    k, v = (pt.gather(c[n][0], c["table"][b], s, page).repeat_interleave(q.shape[1] // Hkv, 0) for n in
            ("k_pages", "v_pages"))                          # [H, s, d]
    x = torch.einsum("nhd,hsd->nhs", q[a:z].double(), k) / math.sqrt(d)
    mag = torch.einsum("nhd,hsd->nhs", q[a:z].double().abs(), k.abs()) / math.sqrt(d)
    p, j = torch.arange(s - (z - a), s)[:, None], torch.arange(s)
    see = (j <= p) & ((j > p - window) | (j < sinks) if window else True)
    x = x.masked_fill(~see[:, None], -math.inf)
    w = torch.softmax(x, -1)
    return (torch.einsum("nhs,hsd->nhd", w, v), torch.logsumexp(x, -1), torch.einsum("nhs,hsd->nhd", w, v.abs()),
            mag.masked_fill(~see[:, None], 0).amax(-1))
