"""The paged cache on the GPU where calls meet one another or go wrong late:
refusals found behind the list's checks, memory of other streams, rows that are
computed again, results that must not depend on what ran before."""

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
