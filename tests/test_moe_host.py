"""Refusals of the sort, dispatch, combine and gradient-norm entry points, struct
layouts and workspace sizes (no GPU: every case returns before the library touches
CUDA)."""
import ctypes
import math
import os
import subprocess

import pytest
import torch

import newton_schulz_02_gb300 as m
from newton_schulz_02_gb300 import build as nbuild
from tests.conftest import ROOT
from tests.test_train_host import Placed, act8, changed, placed

OK, INVALID, MISALIGNED, UNSUPPORTED, SMALL = (m.MUON_OK, m.MUON_ERR_INVALID_ARG, m.MUON_ERR_MISALIGNED,
                                               m.MUON_ERR_UNSUPPORTED, m.MUON_ERR_WORKSPACE_TOO_SMALL)
R = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    nbuild.build()
    return m.load_library()


def test_struct_layouts_match_c(tmp_path):
    structs = ["muon_routing_t", "muon_grads_t"]
    lines = [f'printf("{s} %zu\\n", sizeof({s}));' for s in structs]
    lines += [f'printf("{s}.{f[0]} %zu\\n", offsetof({s}, {f[0]}));'
              for s in structs for f in getattr(m, s)._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "muon.h"\nint main(void){'
                   + "".join(lines) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    for line in subprocess.check_output([str(exe)], text=True).splitlines():
        key, val = line.split()
        s, _, f = key.partition(".")
        got = getattr(getattr(m, s), f).offset if f else ctypes.sizeof(getattr(m, s))
        assert got == int(val), key


def routing(**kw):
    return changed(m.muon_routing_t(10, 8, 4, 2, 0x10000, 0x20000, 0x30000), **kw)


BAD_ROUTING = (dict(tokens=-1), dict(rows=-1), dict(experts=0), dict(topk=0), dict(place=None))
BIG_ROUTING = (dict(experts=1025), dict(topk=1025), dict(tokens=1 << 30), dict(rows=1 << 31))


def test_sort_refusals(lib):
    need = m.muon_moe_sort_workspace_size(10, 4, 2)

    def sort(r=routing(), chosen=0x40000, size=8, stride=2, mask=None, ws=0x100000, n=need):
        return lib.muon_moe_sort(chosen, size, stride, mask, None if r is None else R(r), ws, n, None)

    for bad in BAD_ROUTING + (dict(offsets=None), dict(order=None)):
        assert sort(routing(**bad)) == INVALID, bad
    for big in BIG_ROUTING:
        assert sort(routing(**big)) == UNSUPPORTED, big
    for bad in (dict(r=None), dict(chosen=None), dict(size=2), dict(stride=1), dict(ws=None)):
        assert sort(**bad) == INVALID, bad
    for bad in (dict(chosen=0x40004), dict(ws=0x100080), dict(r=routing(place=0x30002)),
                dict(r=routing(order=0x20001)), dict(r=routing(offsets=0x10003))):
        assert sort(**bad) == MISALIGNED, bad
    assert sort(n=need - 1) == SMALL
    assert lib.muon_moe_sort_workspace_size(10, 4, 2, None) == INVALID
    with pytest.raises(m.MuonError):
        m.muon_moe_sort_workspace_size(1, 2000, 1)


def test_sort_refuses_choices_and_masks_that_share_memory_with_its_outputs(lib):
    """offsets, order and place are [0x10000, 0x10014), [0x20000, 0x20020), [0x30000,
    0x30050).  A workspace that is too small ends the calls that are in order."""
    def sort(chosen, size=4, stride=2, mask=None, **kw):
        return lib.muon_moe_sort(chosen, size, stride, mask, R(routing(**kw)), 0x100000, 0, None)

    for chosen in (0x10000, 0x20000, 0x30000, 0x2001C, 0x10010, 0x3004C, 0x20000 - 0x4C, 0x30000 - 0x4C):
        assert sort(chosen) == INVALID, hex(chosen)
    for chosen in (0x10014, 0x20020, 0x30050, 0x10000 - 0x50, 0x20000 - 0x50, 0x30000 - 0x50):
        assert sort(chosen) == SMALL, hex(chosen)
    assert sort(0x30000 - 0x98, size=8) == INVALID and sort(0x30000 - 0xA0, size=8) == SMALL
    # rows apart: the outputs may lie between two of them
    assert sort(0x1FFF8, stride=16) == SMALL and sort(0x1FFF8, stride=8) == INVALID
    assert sort(0x20000 - 9 * 64 - 4, stride=16) == INVALID and sort(0x20000 - 9 * 64 - 8, stride=16) == SMALL
    assert sort(0x30000 - 8, stride=1 << 62) == SMALL and sort(0x30000 - 4, stride=1 << 62) == INVALID
    for mask in (0x10013, 0x2001F, 0x3004F, 0x20000 - 9, 0x30000 - 9):
        assert sort(0x40000, mask=mask) == INVALID, hex(mask)
    for mask in (0x10014, 0x20020, 0x30050, 0x20000 - 10, 0x30000 - 10):
        assert sort(0x40000, mask=mask) == SMALL, hex(mask)
    assert sort(0x30000, tokens=0) == SMALL and sort(0x20000, rows=0) == SMALL


@pytest.mark.parametrize("tokens,experts,topk", [(1, 1, 1), (4096, 8, 2), (4097, 8, 2), (131072, 256, 8),
                                                 (1 << 21, 1024, 8), (2 ** 31 - 1, 64, 1)])
def test_sort_workspace_is_one_row_of_counts_a_block(lib, tokens, experts, topk):
    """At most 152 blocks, however many copies there are."""
    size = m.muon_moe_sort_workspace_size(tokens, experts, topk)
    assert 256 <= size <= 256 + 1024 + 152 * (experts + 3) * 4


def test_row_pass_refusals(lib):
    x, y, z, w, dw = 0x40000, 0x50000, 0x60000, 0x70000, 0x80000

    def dispatch(r=routing(), x=x, xdt=1, xst=100, width=100, y=y, ydt=0, yst=100, x8=None):
        return lib.muon_moe_dispatch(x, xdt, xst, R(r), width, y, ydt, yst, x8 and R(x8), None)

    def dispatch_b(r=routing(), x=x, xdt=1, xst=100, width=100, y=y, ydt=0, yst=100, acc=0):
        return lib.muon_moe_dispatch_backward(y, ydt, yst, R(r), width, x, xdt, xst, acc, None)

    def combine(r=routing(), x=x, xdt=1, xst=100, width=100, y=y, ydt=0, yst=100, acc=0, w=w, wdt=1, wst=2):
        return lib.muon_moe_combine(y, ydt, yst, R(r), w, wdt, wst, width, x, xdt, xst, acc, None)

    def combine_b(r=routing(), x=x, xdt=1, xst=100, width=100, y=y, ydt=0, yst=100, w=w, wdt=1, wst=2,
                  z=z, zst=100, dw=dw, dwst=2):
        return lib.muon_moe_combine_backward(x, xdt, xst, y, ydt, yst, R(r), w, wdt, wst, width, z, zst,
                                             dw, dwst, None)

    for f in (dispatch, dispatch_b, combine, combine_b):
        for bad in BAD_ROUTING:
            assert f(routing(**bad)) == INVALID, (f, bad)
        for big in BIG_ROUTING:
            assert f(routing(**big)) == UNSUPPORTED, (f, big)
        for bad in (dict(x=None), dict(y=None), dict(xdt=2), dict(ydt=-1), dict(xst=99), dict(yst=99),
                    dict(width=0)):
            assert f(**bad) == INVALID, (f, bad)
        for bad in (dict(x=x + 2), dict(y=y + 1), dict(r=routing(place=0x30001))):
            assert f(**bad) == MISALIGNED, (f, bad)
        assert f(width=(1 << 26) + 1, xst=1 << 30, yst=1 << 30) == UNSUPPORTED
    for f in (combine, combine_b):
        for bad in (dict(w=None), dict(wdt=3), dict(wst=1)):
            assert f(**bad) == INVALID, (f, bad)
        assert f(w=w + 2) == MISALIGNED
    for f in (dispatch_b, combine):
        assert f(acc=2) == INVALID
    for bad in (dict(z=None), dict(zst=99), dict(dw=None), dict(dwst=1)):
        assert combine_b(**bad) == INVALID, bad
    assert combine_b(z=z + 1) == MISALIGNED and combine_b(dw=dw + 2) == MISALIGNED
    assert combine_b(z=y, zst=104) == INVALID     # ys itself, but not its rows
    for bad in (act8(rows=7), act8(cols=99), act8(codes=None)):
        assert dispatch(x8=bad) == INVALID
    assert dispatch(x8=act8(exps=0x20001)) == MISALIGNED
    # no tokens: nothing is enqueued
    none = routing(tokens=0, rows=0, place=None, offsets=None, order=None)
    assert dispatch(none, x=None, y=None) == OK and combine(none, x=None, y=None, w=None) == OK
    assert dispatch_b(none, x=None, y=None) == OK
    assert combine_b(none, x=None, y=None, w=None, z=None, dw=None) == OK


def grads(**kw):
    return changed(m.muon_grads_t(2, 16, 64, 64, m.MUON_BF16, 0x10000), **kw)


def test_grad_norm_refusals(lib):
    nb = ctypes.c_size_t()
    assert lib.muon_grad_norm_workspace_size(R(grads()), 1, R(nb)) == OK

    def call(g=grads(), n=1, most=1.0, norm=0x20000, scale=0x30000, ws=0x100000, size=nb.value):
        return lib.muon_grad_norm(g if g is None else R(g), n, most, norm, scale, ws, size, None)

    for bad in (dict(count=-1), dict(rows=-1), dict(cols=-1), dict(dtype=2), dict(ptrs=None),
                dict(row_stride=63)):
        assert call(grads(**bad)) == INVALID, bad
        assert lib.muon_grad_norm_workspace_size(R(grads(**bad)), 1, R(nb)) == INVALID
    assert call(grads(ptrs=0x10004)) == MISALIGNED and call(grads(row_stride=68)) == MISALIGNED
    assert call(grads(cols=60, row_stride=64)) == UNSUPPORTED
    assert call(grads(rows=1 << 60, row_stride=64)) == UNSUPPORTED
    for bad in (dict(n=-1), dict(g=None), dict(most=-1.0), dict(most=math.nan), dict(norm=None),
                dict(scale=None), dict(ws=None)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(norm=0x20002), dict(scale=0x30001), dict(ws=0x100010)):
        assert call(**bad) == MISALIGNED, bad
    assert call(size=nb.value - 1) == SMALL
    assert lib.muon_grad_norm_workspace_size(R(grads()), 1, None) == INVALID


def test_steps_refuse_a_factor_off_its_boundary(lib):
    g = m.muon_group_t(1, m.muon_view_t(64, 64, 64, 0, 0), 0, 0, 0x10000, 0x10100, 0x10200, None)
    hp, nb = m.hparams(), ctypes.c_size_t()
    assert lib.muon_step_workspace_size(R(g), 1, None, R(nb)) == OK
    assert lib.muon_step_batched_scaled(R(g), 1, R(hp), None, 0x20002, 0x100000, nb.value, None) == MISALIGNED
    a = m.muon_adamw_group_t(1, 8, 0, 0, 0x10000, 0x10100, 0x10200, 0x10300, None)
    ahp = m.adamw_hparams()
    assert lib.muon_adamw_step_scaled(R(a), 1, R(ahp), 0x20002, None, None) == MISALIGNED


# ---- the binding ------------------------------------------------------------
def routing_on(gpu, tokens=4, topk=2, experts=3, rows=8):
    P, i32 = placed, torch.int32
    return m.Routing(P(gpu, experts + 1, dtype=i32), P(gpu, rows, dtype=i32), P(gpu, tokens, topk, dtype=i32))


def test_binding_refuses_operands_of_several_gpus(lib, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    P, i32, u8 = placed, torch.int32, torch.uint8

    def plan(a=0, b=0, c=0):
        m.Routing(P(a, 4, dtype=i32), P(b, 8, dtype=i32), P(c, 4, 2, dtype=i32))

    def sort(r=0, chosen=0, mask=0, ws=0):
        m.muon_moe_sort(P(chosen, 4, 2, dtype=i32), routing_on(r), P(ws, 4096, dtype=u8),
                        mask=P(mask, 4, dtype=u8), stream=0)

    def dispatch(r=0, x=0, xs=0, x8=0):
        a = m.Act8(P(x8, 8, 96, dtype=torch.int8), P(x8, 8, 16, dtype=u8), 70)
        m.muon_moe_dispatch(P(x, 4, 70), routing_on(r), P(xs, 8, 70), a, stream=0)

    def dispatch_b(r=0, dxs=0, dx=0):
        m.muon_moe_dispatch_backward(P(dxs, 8, 70), routing_on(r), P(dx, 4, 70), stream=0)

    def combine(r=0, ys=0, w=0, out=0):
        m.muon_moe_combine(P(ys, 8, 70), P(w, 4, 2), routing_on(r), P(out, 4, 70), stream=0)

    def combine_b(r=0, dout=0, ys=0, w=0, dys=0, dw=0):
        m.muon_moe_combine_backward(P(dout, 4, 70), P(ys, 8, 70), P(w, 4, 2), routing_on(r), P(dys, 8, 70),
                                    P(dw, 4, 2), stream=0)

    for call in (plan, sort, dispatch, dispatch_b, combine, combine_b):
        names = call.__code__.co_varnames[:call.__code__.co_argcount]
        for n in names:
            with pytest.raises(ValueError, match="GPU"):
                call(**{n: 1})
        if call is not plan:
            with pytest.raises(ValueError, match="current device"):
                call(**{n: 1 for n in names})


def test_binding_refuses_shapes_and_types(lib, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    P, i32 = (lambda *s, **k: placed(0, *s, **k)), torch.int32
    r = routing_on(0)

    def turned(*s, **k):
        t = P(*s, **k).t()
        t.gpu = 0
        return t

    with pytest.raises(ValueError, match="GPU"):
        m.Routing.empty(4, 2, 3, device="cpu")
    for bad in ((P(4, dtype=torch.int64), P(8, dtype=i32), P(4, 2, dtype=i32)),
                (P(4, dtype=i32), P(8), P(4, 2, dtype=i32)), (P(4, dtype=i32), P(8, dtype=i32), P(8, dtype=i32)),
                (P(4, dtype=i32), P(8, dtype=i32), turned(2, 4, dtype=i32))):
        with pytest.raises(ValueError):
            m.Routing(*bad)
    ws, h = P(4096, dtype=torch.uint8), torch.float16
    for bad in (lambda: m.muon_moe_sort(P(4, 3, dtype=i32), r, ws, stream=0),
                lambda: m.muon_moe_sort(P(4, 2), r, ws, stream=0),
                lambda: m.muon_moe_sort(P(4, 2, dtype=i32), r, ws, mask=P(3, dtype=torch.bool), stream=0),
                lambda: m.muon_moe_sort(P(4, 2, dtype=i32), r, ws, mask=P(4), stream=0),
                lambda: m.muon_moe_dispatch(P(4, 70, dtype=h), r, P(8, 70), stream=0),
                lambda: m.muon_moe_dispatch(P(5, 70), r, P(8, 70), stream=0),
                lambda: m.muon_moe_dispatch(P(4, 70), r, P(7, 70), stream=0),
                lambda: m.muon_moe_dispatch(P(4, 70), r, P(8, 71), stream=0),
                lambda: m.muon_moe_dispatch(turned(70, 4), r, P(8, 70), stream=0),
                lambda: m.muon_moe_dispatch_backward(P(9, 70), r, P(4, 70), stream=0),
                lambda: m.muon_moe_combine(P(8, 70), P(4, 3), r, P(4, 70), stream=0),
                lambda: m.muon_moe_combine(P(8, 70), P(4, 2, dtype=h), r, P(4, 70), stream=0),
                lambda: m.muon_moe_combine_backward(P(4, 70), P(8, 70), P(4, 2), r,
                                                    P(8, 70, dtype=torch.bfloat16), P(4, 2), stream=0),
                lambda: m.muon_moe_combine_backward(P(4, 70), P(8, 70), P(4, 2), r, P(8, 70),
                                                    P(4, 2, dtype=torch.bfloat16), stream=0)):
        with pytest.raises(ValueError):
            bad()


def test_gradient_list_refuses_what_it_cannot_hold(lib):
    with pytest.raises(ValueError, match="no gradients"):
        m.Grads([])
    with pytest.raises(ValueError, match="GPU"):
        m.Grads([torch.zeros(8)])
    off = torch.zeros(9)[1:].as_subclass(Placed)
    off.gpu = 0
    with pytest.raises(ValueError, match="aligned"):
        m.Grads([off])
    t = [[torch.zeros(8)] for _ in range(4)]
    with pytest.raises(ValueError, match="GPU"):
        m.Grads(m.adamw_groups(*t))
    with pytest.raises(ValueError, match="grad_scale"):
        m.muon_adamw_step(m.adamw_groups(*t), m.adamw_hparams(), grad_scale=torch.ones(1))
