"""Refusals of the balance, checkpoint, gated-activation and weight-gradient
entry points, struct layouts and workspace sizes (no GPU: every case returns
before the library touches CUDA)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import newton_schulz_02_gb300 as m
from newton_schulz_02_gb300 import build as nbuild
from tests.conftest import ROOT

INVALID, MISALIGNED, UNSUPPORTED, SMALL = (m.MUON_ERR_INVALID_ARG, m.MUON_ERR_MISALIGNED,
                                           m.MUON_ERR_UNSUPPORTED, m.MUON_ERR_WORKSPACE_TOO_SMALL)


@pytest.fixture(scope="module")
def lib():
    nbuild.build()
    return m.load_library()


def test_struct_layouts_match_c(tmp_path):
    structs = ["muon_balance_t", "muon_act8_t", "muon_weight_grad_t"]
    lines = [f'printf("{s} %zu\\n", sizeof({s}));' for s in structs]
    lines += [f'printf("{s}.{f[0]} %zu\\n", offsetof({s}, {f[0]}));'
              for s in structs for f in getattr(m, s)._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "muon.h"\nint main(void){'
                   + "".join(lines) + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                           str(exe)])
    for line in subprocess.check_output([str(exe)], text=True).splitlines():
        key, val = line.split()
        s, _, f = key.partition(".")
        got = getattr(getattr(m, s), f).offset if f else ctypes.sizeof(getattr(m, s))
        assert got == int(val), key


def changed(c, **kw):
    d = type(c).from_buffer_copy(c)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def balance(**kw):
    b = m.muon_balance_t(100, 16, 2, 0x10000, m.MUON_BF16, 16, 0x20000, 4, 2, 3, 0x30000, None,
                         m.MUON_SCORE_SOFTMAX, 0.01)
    return changed(b, **kw)


def test_balance_refusals(lib):
    need = m.muon_balance_workspace_size(100, 16, 3)

    def fwd(b, loss=0x40000, counts=0x50000, load=0x60000, ws=0x100000, n=need):
        return lib.muon_balance_forward(ctypes.byref(b), loss, counts, load, ws, n, None)

    def bwd(b, load=0x60000, dloss=None, dl=0x70000, ddt=m.MUON_BF16, stride=16, acc=0):
        return lib.muon_balance_backward(ctypes.byref(b), load, dloss, dl, ddt, stride, acc, None)

    for bad in (dict(tokens=-1), dict(experts=0), dict(sequences=0), dict(dtype=7), dict(score=2),
                dict(logits_stride=15), dict(logits=None), dict(seq_begin=None)):
        assert fwd(balance(**bad)) == INVALID and bwd(balance(**bad)) == INVALID, bad
    for bad in (dict(topk=0), dict(topk=17), dict(chosen_bytes=2), dict(chosen_stride=1),
                dict(chosen=None), dict(coef=float("nan"))):
        assert fwd(balance(**bad)) == INVALID, bad
    for big in (dict(experts=1025, logits_stride=1025), dict(tokens=1 << 31)):
        assert fwd(balance(**big)) == UNSUPPORTED and bwd(balance(**big), stride=2000) == UNSUPPORTED
    assert fwd(balance(), loss=None) == INVALID and fwd(balance(), load=None) == INVALID
    assert fwd(balance(), counts=None) == INVALID and fwd(balance(), ws=None) == INVALID
    assert fwd(balance(), ws=0x100010) == MISALIGNED and fwd(balance(), n=need - 1) == SMALL
    assert fwd(balance(logits=0x10001)) == MISALIGNED and fwd(balance(chosen=0x20002)) == MISALIGNED
    assert fwd(balance(seq_begin=0x30002)) == MISALIGNED
    assert bwd(balance(), ddt=5) == INVALID and bwd(balance(), acc=2) == INVALID
    assert bwd(balance(), stride=15) == INVALID and bwd(balance(), dl=None) == INVALID
    assert bwd(balance(), dl=0x70001) == MISALIGNED and bwd(balance(), dloss=0x70002) == MISALIGNED
    assert lib.muon_balance_forward(None, 0, 0, 0, 0, 0, None) == INVALID
    # a backward pass over no tokens enqueues nothing
    assert bwd(balance(tokens=0, logits=None, chosen=None), dl=None) == m.MUON_OK
    assert lib.muon_balance_workspace_size(10, 4, 1, None) == INVALID


def act8(**kw):
    return changed(m.muon_act8_t(8, 100, 0x10000, 128, 0x20000, 16), **kw)


def test_act8_refusals(lib):
    r = ctypes.byref
    pack = lambda a, x=0x40000, dt=m.MUON_BF16, s=100: lib.muon_act8_pack(x, dt, s, r(a), None)
    unpack = lambda a, x=0x40000, dt=m.MUON_BF16, s=100: lib.muon_act8_unpack(r(a), x, dt, s, None)
    for f in (pack, unpack):
        for bad in (dict(rows=-1), dict(cols=0), dict(code_stride=96), dict(codes=None),
                    dict(exps=None), dict(exp_stride=3)):
            assert f(act8(**bad)) == INVALID, bad
        for bad in (dict(code_stride=130), dict(exp_stride=17), dict(codes=0x10008),
                    dict(exps=0x20004)):
            assert f(act8(**bad)) == MISALIGNED, bad
        assert f(act8(), dt=3) == INVALID and f(act8(), s=99) == INVALID
        assert f(act8(), x=None) == INVALID and f(act8(), x=0x40001) == MISALIGNED
        assert f(act8(cols=(1 << 26) + 1, code_stride=1 << 27, exp_stride=1 << 22)) == UNSUPPORTED
        assert f(act8(rows=0, codes=None, exps=None), x=None) == m.MUON_OK


def test_swiglu_refusals(lib):
    r = ctypes.byref

    def fwd(g8=act8(), u8=act8(), gate=0x40000, up=0x50000, h=0x60000, gs=100, us=100, hs=100, dt=0):
        return lib.muon_act8_swiglu_forward(gate, gs, up, us, dt, h, hs, r(g8), r(u8), None)

    def bwd(g8=act8(), u8=act8(), h8=act8(), dh=0x40000, dg=0x50000, du=0x60000, s=100, dt=0):
        return lib.muon_act8_swiglu_backward(dh, s, dt, r(g8), r(u8), dg, 100, du, 100,
                                             None if h8 is None else r(h8), None)

    for bad in (dict(g8=act8(rows=7)), dict(u8=act8(cols=99)), dict(dt=2), dict(g8=act8(codes=None))):
        assert fwd(**bad) == INVALID and bwd(**bad) == INVALID, bad
    for bad in (dict(gate=None), dict(up=None), dict(h=None), dict(gs=99), dict(us=0), dict(hs=-1)):
        assert fwd(**bad) == INVALID, bad
    for bad in (dict(dh=None), dict(dg=None), dict(du=None), dict(s=99), dict(h8=act8(rows=9)),
                dict(h8=act8(exps=None))):
        assert bwd(**bad) == INVALID, bad
    assert fwd(h=0x60001) == MISALIGNED and bwd(du=0x60001) == MISALIGNED
    assert bwd(u8=act8(exps=0x20001)) == MISALIGNED
    none = act8(rows=0, codes=None, exps=None)
    assert fwd(none, none, None, None, None) == m.MUON_OK
    assert bwd(none, none, None, None, None, None) == m.MUON_OK


def test_weight_grad_refusals(lib):
    base = m.muon_weight_grad_t(8, 64, 2, 0x40000, m.MUON_BF16, 64, act8(), 0x50000, None, 0x60000,
                                6400, 100, m.MUON_BF16, 0)
    nb = ctypes.c_size_t()
    assert lib.muon_act8_weight_grad_workspace_size(ctypes.byref(base), ctypes.byref(nb)) == m.MUON_OK

    def call(ws=0x100000, n=nb.value, **kw):
        return lib.muon_act8_weight_grad(ctypes.byref(changed(base, **kw)), ws, n, None)

    for bad in (dict(rows=-1), dict(out=0), dict(experts=0), dict(dy_dtype=2), dict(g_dtype=9),
                dict(rows=9), dict(dy=None), dict(dy_stride=63), dict(g_stride=99),
                dict(accumulate=2), dict(offsets=None), dict(g_base=None),
                dict(x=act8(codes=None)), dict(x=act8(code_stride=96)), dict(x=act8(exp_stride=3))):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dy=0x40001), dict(offsets=0x50002), dict(g_base=0x60001),
                dict(x=act8(codes=0x10004)), dict(x=act8(exp_stride=20)), dict(g_ptrs=0x70004)):
        assert call(**bad) == MISALIGNED, bad
    assert call(ws=None) == INVALID and call(ws=0x100010) == MISALIGNED
    assert call(n=nb.value - 1) == SMALL
    assert call(experts=70000) == UNSUPPORTED
    assert lib.muon_act8_weight_grad(None, 0x100000, 256, None) == INVALID
    assert lib.muon_act8_weight_grad_workspace_size(ctypes.byref(base), None) == INVALID


def test_binding_refusals(lib):
    """What the binding itself refuses, on CPU tensors (nothing is enqueued)."""
    z = torch.zeros
    with pytest.raises(ValueError):
        m.Balance(z(4, 8, dtype=torch.float16), z(4, 2, dtype=torch.int64))
    with pytest.raises(ValueError):
        m.Balance(z(4, 8), z(3, 2, dtype=torch.int64))
    with pytest.raises(ValueError):
        m.Balance(z(4, 8), z(4, 2, dtype=torch.int16))
    with pytest.raises(ValueError):
        m.Balance(z(8, 4).t(), z(4, 2, dtype=torch.int64))
    with pytest.raises(ValueError):
        m.Balance(z(4, 8), z(4, 2, dtype=torch.int64), mask=z(5, dtype=torch.bool))
    with pytest.raises(ValueError):
        m.Balance(z(4, 8), z(4, 2, dtype=torch.int64), seq_begin=z(3))
    a = m.act8_empty(4, 70, device="cpu")
    assert a.codes.shape == (4, 96) and a.exps.shape == (4, 16) and a.shape == (4, 70)
    with pytest.raises(ValueError):
        m.muon_act8_pack(z(4, 71), a, stream=0)
    with pytest.raises(ValueError):
        m.muon_act8_pack(z(4, 70, dtype=torch.float64), a, stream=0)
    with pytest.raises(ValueError):
        m.muon_act8_swiglu_forward(z(4, 70), z(4, 70, dtype=torch.bfloat16), z(4, 70), a, a, stream=0)
    with pytest.raises(ValueError):
        m.Act8(z(4, 96, dtype=torch.uint8), a.exps, 70)
    with pytest.raises(ValueError):
        m.Act8(a.codes, a.exps, 97)
    ws = z(512, dtype=torch.uint8)
    with pytest.raises(ValueError):
        m.muon_act8_weight_grad(z(4, 8), a, z(2, 8, 71), ws, stream=0)
    with pytest.raises(ValueError):
        m.muon_act8_weight_grad(z(3, 8), a, z(2, 8, 70), ws, stream=0)
    with pytest.raises(ValueError):
        m.muon_act8_weight_grad(z(4, 8), a, z(2, 8, 70), ws, stream=0,
                                offsets=z(2, dtype=torch.int32))


def test_checkpoint_needs_whole_blocks(lib):
    """A pass writes whole blocks of 32 codes: a view that ends inside one would have
    its neighbours overwritten, or what lies behind its tensor."""
    big, exps = torch.zeros(4, 192, dtype=torch.int8), torch.zeros(4, 16, dtype=torch.uint8)
    for width, cols in ((70, 70), (95, 70), (31, 1), (33, 33)):
        with pytest.raises(ValueError, match="whole blocks"):
            m.Act8(big[:, :width], exps, cols)
    with pytest.raises(ValueError):
        m.Act8(big[:, :96], exps[:, :2], 70)
    for width, cols in ((96, 70), (32, 1), (64, 33), (192, 192)):
        assert m.Act8(big[:, :width], exps[:, :(cols + 31) // 32], cols).c.code_stride == 192


def test_checkpoint_of_one_row(lib):
    """One row cut out of a checkpoint is as good as several: the stride between rows
    that are not there does not matter."""
    codes, exps = torch.zeros(8, 192, dtype=torch.int8), torch.zeros(8, 16, dtype=torch.uint8)
    for n in (0, 1, 2):
        c = m.Act8(codes[3:3 + n, :72 + 24], exps[3:3 + n, :3], 72).c
        assert c.code_stride % 32 == 0 and c.code_stride >= 96 and c.exp_stride % 16 == 0
        assert c.codes == codes.data_ptr() + 3 * 192 or n == 0
    one = m.Act8(torch.zeros(1, 100, dtype=torch.int8), torch.zeros(1, 3, dtype=torch.uint8), 72).c
    assert (one.code_stride, one.exp_stride) == (96, 16)


@pytest.mark.parametrize("experts,blocks", [(8, 5), (64, 5), (200, 5), (512, 5), (513, 2), (1024, 2)])
@pytest.mark.parametrize("sequences", [1, 32, 300])
def test_balance_chunks_fill_one_wave(lib, experts, blocks, sequences):
    """A chunk leaves one row of partial sums and one of counts: as many as one wave
    of blocks on 152 SMs, or half of one beside the sequences' own."""
    size = m.muon_balance_workspace_size(1 << 20, experts, sequences)
    chunks = (size - 4 * sequences * ((experts + 31) // 32)) / (8 * experts + 8)
    padding = 6 * 256 / (8 * experts + 8) + 1
    wave = 152 * blocks
    assert chunks <= max(wave, wave // 2 + sequences) + padding
    assert chunks >= 0.97 * min(wave, wave // 2 + sequences) - padding


class Placed(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""

    def get_device(self):
        return self.gpu

    @property
    def is_cuda(self):
        return True


def placed(gpu, *shape, dtype=torch.float32):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(Placed)
    t.gpu = gpu
    return t


def test_binding_refuses_operands_of_several_gpus(lib, monkeypatch):
    """Every operand on the first one's GPU, and that the current one (no call gets
    as far as the library: there is no GPU here)."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    P, i32, i64, u8 = placed, torch.int32, torch.int64, torch.uint8

    def act8(gpu):
        return m.Act8(P(gpu, 4, 96, dtype=torch.int8), P(gpu, 4, 16, dtype=u8), 70)

    def bal(a=0, b=0, c=0, d=0):
        return m.Balance(P(a, 4, 8), P(b, 4, 2, dtype=i64), P(c, 2, dtype=i32), P(d, 4, dtype=u8))

    def fwd(b=0, loss=0, counts=0, load=0, ws=0):
        m.muon_balance_forward(bal(b, b, b, b), P(loss, 1), P(counts, 8, dtype=i32), P(load, 1, 8),
                               P(ws, 4096, dtype=u8), stream=0)

    def bwd(b=0, load=0, dl=0, dloss=0):
        m.muon_balance_backward(bal(b, b, b, b), P(load, 1, 8), P(dl, 4, 8), P(dloss, 1), stream=0)

    def swf(x=0, y=0, z=0, g=0, u=0):
        m.muon_act8_swiglu_forward(P(x, 4, 70), P(y, 4, 70), P(z, 4, 70), act8(g), act8(u), stream=0)

    def swb(x=0, y=0, z=0, g=0, u=0, h=0):
        m.muon_act8_swiglu_backward(P(x, 4, 70), act8(g), act8(u), P(y, 4, 70), P(z, 4, 70), act8(h), stream=0)

    def wg(dy=0, x=0, G=0, ws=0, off=0):
        m.muon_act8_weight_grad(P(dy, 4, 8), act8(x), P(G, 2, 8, 70), P(ws, 1 << 16, dtype=u8),
                                offsets=P(off, 3, dtype=i32), stream=0)

    def pack(x=0, a=0):
        m.muon_act8_pack(P(x, 4, 70), act8(a), stream=0)

    def unpack(x=0, a=0):
        m.muon_act8_unpack(act8(a), P(x, 4, 70), stream=0)

    for call in (bal, fwd, bwd, swf, swb, wg, pack, unpack):
        names = call.__code__.co_varnames[:call.__code__.co_argcount]
        for n in names:
            with pytest.raises(ValueError, match="GPU"):
                call(**{n: 1})
        if call is not bal:   # all on a GPU that is not the current one
            with pytest.raises(ValueError, match="current device"):
                call(**{n: 1 for n in names})
    assert m.Act8(P(0, 4, 96, dtype=torch.int8), P(1, 4, 16, dtype=u8), 70).ref is None
    bal()


def test_binding_refuses_host_memory(lib):
    """Tensors of the CPU, right in everything else (nothing is enqueued)."""
    z = torch.zeros
    with pytest.raises(ValueError, match="GPU"):
        m.Balance(z(4, 8), z(4, 2, dtype=torch.int64))
    a = m.act8_empty(4, 70, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        m.muon_act8_pack(z(4, 70), a, stream=0)
    with pytest.raises(ValueError, match="GPU"):
        m.muon_act8_unpack(a, z(4, 70), stream=0)
    with pytest.raises(ValueError, match="GPU"):
        m.muon_act8_swiglu_forward(z(4, 70), z(4, 70), z(4, 70), a, a, stream=0)
    with pytest.raises(ValueError, match="GPU"):
        m.muon_act8_weight_grad(z(4, 8), a, z(1, 8, 70), z(512, dtype=torch.uint8), stream=0)
    assert a.ref is None and m.Act8(a.codes, a.exps, 70).ref is None   # a call takes it as a missing argument


def test_operands_of_the_other_cta_are_released_at_cluster_scope():
    """The MMAs that one CTA of a pair issues read the other's shared memory: what
    tells the issuer's barrier of it has to release at cluster scope (a CTA-scope
    release does not pair with the issuer's cluster-scope acquire), as an arrival
    that says so or as the completion of an asynchronous store."""
    with open(os.path.join(nbuild.CSRC, "act8_wgrad.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    remote = re.findall(r"(\w+)\s*=\s*mapa_shared\(&ready\b", code) + [r"mapa_shared\(&ready"]
    names = "(?:" + "|".join(remote) + ")"
    assert not re.search(rf"mbar_arrive_cluster\(\s*{names}", code)
    assert re.search(rf"(mbar_arrive_release_cluster\(|st_async_cluster\([^;]*,)\s*{names}", code)
    assert re.search(r"wait_cluster\(&ready\b", code)
