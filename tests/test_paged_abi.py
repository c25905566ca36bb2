"""The paged cache's C boundary without a GPU: struct layouts, workspace sizes,
and the calls that are refused before anything is launched."""

import ctypes
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000   # never dereferenced: every case fails on the host first


@pytest.fixture(scope="module")
def paged():
    from gated_linear_sliding_chunkwise_b200 import build
    build.build()
    from gated_linear_sliding_chunkwise_b200 import paged
    return paged


@pytest.fixture(scope="module")
def lz(paged):
    from gated_linear_sliding_chunkwise_b200 import lizard
    return lizard


def test_struct_layouts_match_c(paged, tmp_path):
    fields = {"lizard_paged_args": paged.PagedArgs, "lizard_pages_args": paged.PagesArgs}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "lizard.h"', "int main(void) {"]
    for cname, py in fields.items():
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines():
        cname, what, val = line.split()
        py = fields[cname]
        assert int(val) == (ctypes.sizeof(py) if what == "size" else getattr(py, what).offset), f"{cname}.{what}"


def test_new_statuses_have_descriptions(lz):
    for code in (lz.ERR_INDEX, lz.ERR_PAGES):
        assert "paged cache" in lz.status_string(code)


def _attn(paged, lz, **over):
    a = paged.PagedArgs()
    a.layers, a.num_pages, a.Hkv, a.page, a.d, a.rows, a.max_pages = 2, 10, 2, 16, 64, 4, 8
    a.B, a.T, a.H, a.layer, a.max_q, a.dtype, a.impl = 3, 7, 4, 1, 3, lz.BF16, lz.IMPL_AUTO
    for n in ("q", "k", "v", "k_pages", "v_pages", "table", "lens", "cu_q", "row", "lse", "workspace"):
        setattr(a, n, FAKE)
    a.o = 2 * FAKE
    a.workspace_bytes = 1 << 40
    for n, x in over.items():
        setattr(a, n, x)
    return a


@pytest.mark.parametrize("over,code", [
    ({"page": 48}, 2), ({"page": 8}, 2), ({"page": 256}, 2), ({"page": 0}, 1), ({"d": 96}, 2), ({"d": 0}, 1),
    ({"num_pages": 0}, 1), ({"num_pages": (1 << 22) + 1}, 2), ({"rows": 0}, 1), ({"max_pages": 0}, 1),
    ({"rows": 1 << 20, "max_pages": 1 << 12}, 2), ({"max_pages": 1 << 27}, 2),
    ({"num_pages": 1 << 22, "Hkv": 32, "H": 32, "page": 128}, 2),
    ({"layers": 0}, 1), ({"layer": 2}, 1), ({"layer": -1}, 1), ({"Hkv": 0}, 1), ({"Hkv": 3}, 1), ({"H": 0}, 1),
    ({"H": 130}, 2), ({"B": -1}, 1), ({"T": -1}, 1), ({"max_q": 0}, 1), ({"max_q": -1}, 1), ({"window": -1}, 1),
    ({"sinks": -1}, 1), ({"dtype": 2}, 1), ({"impl": 3}, 1), ({"impl": 2, "dtype": 1}, 2),
    ({"softmax_scale": -1.0}, 1), ({"softmax_scale": float("nan")}, 1), ({"softmax_scale": float("inf")}, 1),
    ({"k": None}, 1), ({"v": None}, 1), ({"q": None}, 1), ({"o": None}, 1), ({"table": None}, 1), ({"lens": None}, 1),
    ({"cu_q": None}, 1), ({"k_pages": None}, 1), ({"v_pages": None}, 1), ({"q": FAKE + 8}, 1), ({"row": FAKE + 4}, 1),
    ({"o": FAKE}, 1), ({"workspace": FAKE + 8}, 1), ({"workspace": None}, 5), ({"workspace_bytes": 100}, 5),
])
def test_attention_refuses_bad_arguments_on_host(paged, lz, over, code):
    assert lz.lib().lizard_paged_attn(ctypes.byref(_attn(paged, lz, **over)), None) == code


def test_workspace_sizes(paged, lz):
    size = lz.lib().lizard_paged_attn_workspace_size
    a = _attn(paged, lz)
    need = size(ctypes.byref(a))
    assert need > 0 and size(None) == 0
    assert size(ctypes.byref(_attn(paged, lz, page=48))) == 0
    for n in ("q", "k", "v", "k_pages", "v_pages", "table", "lens", "cu_q", "row", "o", "lse", "workspace"):
        setattr(a, n, None)
    assert size(ctypes.byref(a)) == need                     # pointers are ignored
    a = _attn(paged, lz, workspace_bytes=need - 1)
    assert lz.lib().lizard_paged_attn(ctypes.byref(a), None) == lz.ERR_WORKSPACE
    psize = lz.lib().lizard_pages_workspace_size
    p = _pages(paged, lz)
    assert psize(ctypes.byref(p)) > 0 and psize(None) == 0
    p.workspace_bytes = psize(ctypes.byref(p)) - 1
    for name in ("reserve", "free", "fork", "compact"):
        assert getattr(lz.lib(), "lizard_pages_" + name)(ctypes.byref(p), None) == lz.ERR_WORKSPACE


def _pages(paged, lz, **over):
    a = paged.PagesArgs()
    a.layers, a.num_pages, a.Hkv, a.page, a.d, a.rows, a.max_pages, a.dtype, a.n = 1, 10, 2, 16, 64, 4, 8, lz.FP32, 3
    for n in ("k_pages", "v_pages", "refs", "table", "lens", "row", "src", "grow", "table_out", "refs_out", "workspace"):
        setattr(a, n, FAKE)
    a.workspace_bytes = 1 << 40
    for n, x in over.items():
        setattr(a, n, x)
    return a


ALL = ("reserve", "free", "fork", "compact")


@pytest.mark.parametrize("over,code,names", [
    ({"page": 24}, 2, ALL), ({"num_pages": 0}, 1, ALL), ({"num_pages": 1 << 23}, 2, ALL), ({"rows": 0}, 1, ALL),
    ({"n": -1}, 1, ALL), ({"n": 5}, 1, ALL), ({"refs": None}, 1, ALL), ({"table": None}, 1, ALL),
    ({"refs": FAKE + 4}, 1, ALL), ({"workspace": None}, 5, ALL),
    ({"lens": None}, 1, ("reserve", "free", "fork")), ({"row": None}, 1, ("reserve", "free", "fork")),
    ({"grow": None}, 1, ("reserve",)), ({"src": None}, 1, ("fork",)),
    ({"d": 32}, 2, ("fork", "compact")), ({"dtype": 5}, 1, ("fork", "compact")), ({"layers": 0}, 1, ("fork", "compact")),
    ({"k_pages": None}, 1, ("fork", "compact")), ({"v_pages": None}, 1, ("fork", "compact")),
    ({"table_out": None}, 1, ("compact",)), ({"refs_out": None}, 1, ("compact",)),
])
def test_bookkeeping_refuses_bad_arguments_on_host(paged, lz, over, code, names):
    for name in names:
        a = _pages(paged, lz, **over)
        assert getattr(lz.lib(), "lizard_pages_" + name)(ctypes.byref(a), None) == code, name


def test_binding_refuses_tensors_that_do_not_fit(paged):
    kp = torch.zeros(1, 4, 2, 16, 64)
    q, k, i = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64), lambda *x: torch.tensor(x, dtype=torch.int32)
    table, lens, cu = torch.zeros(2, 2, dtype=torch.int32), i(3, 3), i(0, 1, 3)
    good = dict(q=q, k=k, v=k, k_pages=kp, v_pages=kp, table=table, lens=lens, cu_q=cu)
    for name, bad in (("q", q.bfloat16()), ("q", torch.zeros(3, 4, 128)), ("q", q.transpose(0, 1)), ("k", q), ("k", None),
                      ("v", k[:2]), ("v_pages", kp.bfloat16()), ("v_pages", kp[:, :3]), ("k_pages", kp[0]),
                      ("table", table.long()), ("table", table[0]), ("lens", i(1)), ("lens", lens.long()),
                      ("cu_q", cu.long()), ("cu_q", i(0, 1, 1, 3)), ("table", torch.zeros(2, 4, dtype=torch.int32)[:, ::2])):
        with pytest.raises(ValueError):
            paged.attn(**{**good, name: bad}, max_q=2)
    with pytest.raises(ValueError):
        paged.attn(**good, max_q=2, row=i(0))
    with pytest.raises(ValueError, match="CUDA"):            # nothing on the host reaches a kernel
        paged.attn(**good, max_q=2)
    with pytest.raises(TypeError):
        paged.attn(**{**good, "q": q.half(), "k": k.half(), "v": k.half(), "k_pages": kp.half(), "v_pages": kp.half()},
                   max_q=2)
    refs = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: paged.reserve(refs.long(), table, lens, i(0), i(1), page=16),
                 lambda: paged.reserve(refs, table, lens, i(0), i(1, 2), page=16),
                 lambda: paged.free(refs, table, i(3), i(0), page=16),
                 lambda: paged.fork(kp, kp, refs[:3], table, lens, i(0), i(1)),
                 lambda: paged.fork(kp, kp, refs, table, lens, i(0, 1), i(1)),
                 lambda: paged.compact(kp, kp, refs, table, table_out=table[:1]),
                 lambda: paged.free(refs, table, lens, i(0), page=16)):
        with pytest.raises(ValueError):
            call()


def test_a_truth_value_that_raises_is_the_callers_error(paged):
    """want_lse's own exception comes through, and nothing is launched."""
    class Undecided:
        def __bool__(self):
            raise ZeroDivisionError("undecided")

    kp, x = torch.zeros(1, 4, 2, 16, 64), torch.zeros(2, 2, 64)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ZeroDivisionError):
        paged.attn(x, x, x, kp, kp, i[:, None].contiguous(), i, torch.zeros(3, dtype=torch.int32), max_q=1,
                   want_lse=Undecided())


def test_compact_takes_any_workspace_that_the_size_query_gives(paged, lz):
    """compact has no list: n counts towards the workspace's size alone, and is checked like the others'."""
    size = lz.lib().lizard_pages_workspace_size
    bytes_of = [size(ctypes.byref(_pages(paged, lz, n=n))) for n in range(5)]
    assert bytes_of == sorted(bytes_of) and bytes_of[0] > 0
    for n in (-1, 5):
        a = _pages(paged, lz, n=n)
        assert size(ctypes.byref(a)) == 0
        assert lz.lib().lizard_pages_compact(ctypes.byref(a), None) == lz.ERR_INVALID_ARG


def test_slices_off_a_16_byte_boundary_are_named(paged):
    """The library wants pointers on 16-byte boundaries: the refusal says which tensor is not."""
    kp, x = torch.zeros(1, 4, 2, 16, 64), torch.zeros(2, 2, 64)
    i = torch.zeros(8, dtype=torch.int32)
    good = dict(q=x, k=x, v=x, k_pages=kp, v_pages=kp, table=i[:8].view(2, 4), lens=i[:2], cu_q=i[:3], row=i[:2])
    for name, bad in (("row", i[1:3]), ("lens", i[3:5]), ("cu_q", i[2:5]), ("table", i[1:7].view(2, 3)),
                      ("q", torch.zeros(300)[1:257].view(2, 2, 64))):
        with pytest.raises(ValueError, match=f"{name} must begin on a 16-byte boundary"):
            paged.attn(**{**good, name: bad}, max_q=1)
    refs, table = torch.zeros(5, dtype=torch.int32), i.view(2, 4)
    with pytest.raises(ValueError, match="refs must begin"):
        paged.free(refs[1:], table, i[:2], i[:1], page=16)
    with pytest.raises(ValueError, match="row must begin"):
        paged.free(refs, table, i[:2], i[1:2], page=16)
    with pytest.raises(ValueError, match="CUDA"):            # an empty slice has no address
        paged.free(refs, table, i[:2], i[1:1], page=16)


@pytest.mark.parametrize("name,heads", [("q", 4), ("k", 2), ("v", 2)])
def test_an_output_over_any_part_of_the_inputs_is_refused(paged, lz, name, heads):
    """o [7, 4, 64] bf16 against q [7, 4, 64], k and v [7, 2, 64], from either end."""
    far = {n: (16 + i) * FAKE for i, n in enumerate(("q", "k", "v"))}
    call, size = lz.lib().lizard_paged_attn, 7 * heads * 64 * 2
    out = 7 * 4 * 64 * 2
    for at, code in ((far[name] + size - 16, lz.ERR_INVALID_ARG), (far[name] - out + 16, lz.ERR_INVALID_ARG),
                     (far[name], lz.ERR_INVALID_ARG), (far[name] + size, lz.ERR_WORKSPACE),
                     (far[name] - out, lz.ERR_WORKSPACE)):
        a = _attn(paged, lz, **far, o=at, workspace_bytes=100)      # the next check behind this one
        assert call(ctypes.byref(a), None) == code
    a = _attn(paged, lz, **far, H=2, o=far[name], workspace_bytes=100)   # as many query heads as the others
    assert call(ctypes.byref(a), None) == (lz.ERR_INVALID_ARG if name == "q" else lz.ERR_WORKSPACE)
