"""Tokens sorted by expert, dispatched and combined, with their gradients, on the
GPU against the float64 oracle (oracle/moe_ref.py).

Numbers of the sort are exact.  Tolerances of the others, U = 2^-24, HALF of a type
half a step relative to the value (bf16 2^-8, fp32 U):
  dispatch   a value is rounded to its row's type once: HALF |x|; checkpoints are
             those that muon_act8_pack writes of the same values, bit for bit.
  combine    at most K products and additions in a chain, and one more when it
             accumulates: (K + 2) U times the sum of the terms' magnitudes; HALF.
  gradients  one product and its rounding: 2 HALF of dys.  dweights: the D products
             are added up in fp32, in whatever order, by at most D additions:
             (D + 2) U times the sum of their magnitudes; HALF."""
import numpy as np
import pytest
import torch

import newton_schulz_02_gb300 as m
from oracle import moe_ref as R
from tests.gpu_util import f64
from tests.test_gpu_train import framed, put, untouched, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": U}


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()
    torch.cuda.set_device(0)


def choices(seed, T, E, K, drop=0.0):
    """Choices of a router that likes some experts more; a token may choose one twice."""
    rng = np.random.default_rng(seed)
    p = rng.random(E) ** 3 + 1e-3
    c = rng.choice(E, size=(T, K), p=p / p.sum())
    c[rng.random((T, K)) < drop] = -1
    return c


def run_sort(chosen, E, mask=None, rows=None, idx=torch.int64, stride=None):
    """(routing, flags) with every output set to a mark before."""
    T, K = chosen.shape
    c = torch.full((T, stride or K), 10 ** 6, dtype=idx, device=DEV)[:, :K]
    c.copy_(torch.as_tensor(chosen))
    r = m.Routing.empty(T, K, E, rows=rows)
    for t in (r.offsets, r.order, r.place):
        t.fill_(-77)
    ws = m.workspace(m.muon_moe_sort_workspace_size(T, E, K))
    ws.fill_(255)
    mk = None if mask is None else torch.as_tensor(mask).to(DEV)
    m.muon_moe_sort(c, r, ws, mask=mk)
    code, flags = m.muon_get_status(ws)
    assert code == m.MUON_OK
    return r, flags


def check_sort(r, flags, chosen, E, mask=None, rows=None):
    offsets, order, place, bad = R.sort(chosen, E, mask, rows)
    assert r.offsets.tolist() == offsets.tolist()
    got = r.order.cpu().numpy()
    assert np.array_equal(got[:len(order)], order)
    assert (got[len(order):] == -77).all()      # rows behind the last stay as they were
    assert np.array_equal(r.place.cpu().numpy(), place)
    assert flags == (m.MUON_FLAG_INDEX if bad else 0)


@pytest.mark.parametrize("T,E,K", [(0, 4, 2), (1, 1, 1), (1, 8, 8), (33, 8, 2), (100, 7, 3), (511, 60, 6),
                                   (1024, 16, 1), (1025, 1024, 8), (4097, 257, 2), (9000, 1000, 1),
                                   (20011, 33, 5)])
@pytest.mark.parametrize("idx", [torch.int32, torch.int64])
def test_sort(T, E, K, idx):
    chosen = choices(T + E, T, E, K, drop=0.1)
    mask = np.random.default_rng(1).random(T) > 0.2
    check_sort(*run_sort(chosen, E, idx=idx), chosen, E)
    check_sort(*run_sort(chosen, E, mask, idx=idx, stride=K + 3), chosen, E, mask)


def test_sort_more_copies_than_a_wave_holds():
    """Blocks of several rounds: 400000 tokens of 4 choices, against a stable sort."""
    T, E, K = 400000, 200, 4
    chosen = torch.as_tensor(choices(5, T, E, K, drop=0.05), device=DEV)
    r = m.Routing.empty(T, K, E)
    r.order.fill_(-77)
    ws = m.workspace(m.muon_moe_sort_workspace_size(T, E, K))
    m.muon_moe_sort(chosen, r, ws)
    key = torch.where(chosen < 0, E, chosen).flatten()
    want = torch.sort(key, stable=True).indices
    n = int((key < E).sum())
    assert r.offsets[-1].item() == n and torch.equal(r.order[:n].long(), want[:n])
    assert bool((r.order[n:] == -77).all())
    assert torch.equal(r.offsets.long(), torch.searchsorted(key[want], torch.arange(E + 1, device=DEV)))
    place = torch.full((T * K,), -1, dtype=torch.int32, device=DEV)
    place[want[:n]] = torch.arange(n, dtype=torch.int32, device=DEV)
    assert torch.equal(r.place.flatten(), place)
    assert m.muon_get_status(ws) == (m.MUON_OK, 0)


@pytest.mark.parametrize("T", [300, 30000])
def test_sort_one_expert_takes_all_and_all_tokens_masked(T):
    one = np.full((T, 3), 5)
    check_sort(*run_sort(one, 9), one, 9)
    none = np.zeros(T, dtype=bool)
    check_sort(*run_sort(one, 9, none), one, 9, none)


@pytest.mark.parametrize("T", [50, 20000])
def test_sort_bad_numbers_and_too_few_rows_are_flagged(T):
    chosen = choices(3, T, 12, 2)
    for bad in (12, -2, 2 ** 31 - 1, -(2 ** 31)):
        c = chosen.copy()
        c[T // 2, 1] = bad
        check_sort(*run_sort(c, 12, idx=torch.int32), c, 12)
    c = chosen.copy()
    c[0, 0] = 2 ** 32 + 3      # its low half is an expert
    check_sort(*run_sort(c, 12), c, 12)
    for rows in (0, 1, T, 2 * T - 1, 2 * T, 2 * T + 5):
        check_sort(*run_sort(chosen, 12, rows=rows), chosen, 12, rows=rows)
    mask = np.ones(T, dtype=bool)
    mask[T // 2] = False       # the choices of masked tokens are not looked at
    c = chosen.copy()
    c[T // 2] = 99
    r, flags = run_sort(c, 12, mask)
    assert flags == 0


def stable_sort(chosen, E, mask, rows):
    """R.sort of many copies at once: (offsets, order, place, bad)."""
    T, K = chosen.shape
    on = np.ones((T, K), dtype=bool) if mask is None else np.repeat(mask[:, None], K, axis=1)
    known = (chosen >= 0) & (chosen < E)
    key = np.where(on & known, chosen, E).ravel()
    n = int((key < E).sum())
    order = np.argsort(key, kind="stable")[:n]
    ends = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
    bad = bool((on & ~known & (chosen != -1)).any()) or n > rows
    order = order[:rows]
    place = np.full(T * K, -1, dtype=np.int64)
    place[order] = np.arange(len(order))
    return np.minimum(ends, rows), order, place.reshape(T, K), bad


# Copies at the borders between the forms: one block of one or two copies a thread (2048),
# blocks of one, two and three to eight copies a thread (up to 155648, 311296, 1245184),
# and several rounds of those.
@pytest.mark.parametrize("T,E,K", [(1025, 9, 1), (2047, 300, 1), (1024, 1024, 2), (683, 60, 3), (19456, 256, 8),
                                   (51883, 31, 3), (38912, 256, 8), (44471, 1000, 7), (65536, 256, 8),
                                   (131071, 256, 8), (131071, 1024, 8), (155648, 64, 8), (249037, 257, 5),
                                   (400000, 128, 8)])
def test_sort_in_each_of_its_forms(T, E, K):
    rng = np.random.default_rng(T + E)
    chosen = choices(T, T, E, K, drop=0.05)
    mask = rng.random(T) > 0.1
    mask[-1] = mask[T // 2] = True
    ways = ((torch.int64, None, None, T * K, None), (torch.int32, K + 3, mask, T * K, None),
            (torch.int64, K + 1, mask, T * K * 2 // 3, None), (torch.int32, None, None, T * K + 3, E),
            (torch.int64, None, mask, T * K // 2 + 1, 2 ** 32 + 3), (torch.int32, K + 2, None, T * K - 1, -2))
    for idx, stride, mk, rows, bad in ways:
        c = chosen.copy()
        if bad is not None:
            c[T // 2 if bad > 0 else -1, K - 1] = bad
        r, flags = run_sort(c, E, mk, rows, idx, stride)
        offsets, order, place, flagged = stable_sort(c, E, mk, rows)
        assert np.array_equal(r.offsets.cpu().numpy(), offsets)
        got = r.order.cpu().numpy()
        assert np.array_equal(got[:len(order)], order) and (got[len(order):] == -77).all()
        assert np.array_equal(r.place.cpu().numpy(), place)
        assert flags == (m.MUON_FLAG_INDEX if flagged else 0)
        if T * K < 2100:
            check_sort(r, flags, c, E, mk, rows)


@pytest.mark.parametrize("T,K,stride", [(2 ** 31 - 1, 1, 1), ((2 ** 31 - 1) // 7, 7, 8)])
def test_sort_of_as_many_copies_as_it_takes(T, K, stride):
    """Copy i chooses expert i mod 5, or none where i mod 5 = 4: its row is i // 5 behind the
    expert's first."""
    E, n = 4, T * K
    chosen = torch.empty(T, stride, dtype=torch.int32, device=DEV)[:, :K]
    step = (1 << 26) // K
    for t in range(0, T, step):     # a part of the tokens at a time
        i = torch.arange(t * K, min(T, t + step) * K, device=DEV)
        e = i % 5
        chosen[t:t + step] = torch.where(e == 4, -1, e).to(torch.int32).view(-1, K)
    r = m.Routing.empty(T, K, E)
    r.order.fill_(-77)
    ws = m.workspace(m.muon_moe_sort_workspace_size(T, E, K))
    m.muon_moe_sort(chosen, r, ws)
    assert m.muon_get_status(ws) == (m.MUON_OK, 0)
    sizes = [(n - e + 4) // 5 for e in range(E)]
    assert r.offsets.tolist() == [sum(sizes[:e]) for e in range(E + 1)]
    first = r.offsets.long()
    for t in range(0, T, step):
        i = torch.arange(t * K, min(T, t + step) * K, device=DEV)
        e = i % 5
        want = torch.where(e == 4, -1, first[e] + i // 5)
        assert torch.equal(r.place[t:t + step].flatten().long(), want)
    for e in range(E):
        for a in range(0, sizes[e], 1 << 26):
            b = min(sizes[e], a + (1 << 26))
            rows = r.order[int(first[e]) + a:int(first[e]) + b]
            assert torch.equal(rows.long(), 5 * torch.arange(a, b, device=DEV) + e)
    assert bool((r.order[int(first[E]):] == -77).all())


# ---- activations ------------------------------------------------------------
def routed(seed, T, E, K, drop=0.15, rows=None):
    chosen = choices(seed, T, E, K, drop)
    r, _ = run_sort(chosen, E, rows=rows)
    return r, r.place.cpu().numpy()


SIZES = [(1, 1, 1, 1), (1, 3, 8, 16), (5, 4, 2, 31), (70, 8, 2, 512), (33, 60, 6, 1111), (19, 16, 9, 77),
         (40, 5, 3, 8), (9, 4, 17, 4100), (6, 3, 2, 8193), (3, 1024, 1024, 40)]
TYPES = [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("outer,inner", TYPES)
@pytest.mark.parametrize("how", ["dense", "padded", "shifted"])
@pytest.mark.parametrize("T,E,K,D", SIZES)
def test_dispatch(outer, inner, how, T, E, K, D):
    r, place = routed(T + D, T, E, K)
    x = put(np.random.default_rng(D).normal(size=(T, D)), DT[outer], how)
    buf, xs = framed(r.rows, D, DT[inner], how)
    x8, alone = m.act8_empty(r.rows, D), m.act8_empty(r.rows, D)
    for a in (x8, alone):
        a.codes.fill_(99)
        a.exps.fill_(98)
    m.muon_moe_dispatch(x, r, xs, x8)
    want = R.dispatch(f64(x), place, r.rows)
    held = ~np.isnan(want[:, 0])
    got = f64(xs)
    within(got[held], want[held], HALF[inner] * np.abs(want[held]))
    assert (got[~held] == 7.0).all() and untouched(buf, xs)
    # the checkpoint: what packing the rows of x writes
    rows = torch.as_tensor(np.where(held)[0], device=DEV)
    source = (r.order[rows].long() // K) if len(rows) else rows
    packed = m.act8_empty(len(rows), D)
    m.muon_act8_pack(x[source].contiguous(), packed)
    nb = (D + 31) // 32
    assert torch.equal(x8.codes[rows], packed.codes) and torch.equal(x8.exps[rows, :nb], packed.exps[:, :nb])
    rest = torch.as_tensor(np.where(~held)[0], device=DEV)
    assert torch.equal(x8.codes[rest], alone.codes[rest]) and torch.equal(x8.exps[rest], alone.exps[rest])
    # without a checkpoint
    buf2, xs2 = framed(r.rows, D, DT[inner], how)
    m.muon_moe_dispatch(x, r, xs2)
    assert torch.equal(buf2, buf)


@pytest.mark.parametrize("outer,inner", TYPES)
@pytest.mark.parametrize("D", [127, 128, 129, 130, 255, 256, 257, 263, 511, 513, 1023, 1025, 1031, 2049])
def test_dispatch_rows_at_every_offset(outer, inner, D):
    """Rows whose stride runs through all offsets from a 16-byte boundary, inside a
    buffer whose every other value has to stay."""
    T, E, K = 5, 3, 4
    r, place = routed(D, T, E, K, drop=0.1)
    x = put(np.random.default_rng(D).normal(size=(T, D)), DT[outer], "shifted")
    want = R.dispatch(f64(x), place, r.rows)
    held = ~np.isnan(want[:, 0])
    for stride, lead in ((D + 1, 0), (D + 3, 1), (D + 2, 2)):
        buf = torch.full((r.rows * stride + 16,), 7.0, dtype=DT[inner], device=DEV)
        xs = buf[lead:].as_strided((r.rows, D), (stride, 1))
        x8 = m.act8_empty(r.rows, D)
        m.muon_moe_dispatch(x, r, xs, x8)
        got = f64(xs)
        within(got[held], want[held], HALF[inner] * np.abs(want[held]))
        assert (got[~held] == 7.0).all() and untouched(buf, xs)
        first = torch.as_tensor(np.where(held)[0], device=DEV)
        packed = m.act8_empty(len(first), D)
        m.muon_act8_pack(x[r.order[first].long() // K].contiguous(), packed)
        nb = (D + 31) // 32
        assert torch.equal(x8.codes[first], packed.codes) and torch.equal(x8.exps[first, :nb], packed.exps[:, :nb])


@pytest.mark.parametrize("outer,inner", TYPES)
@pytest.mark.parametrize("how", ["dense", "padded", "shifted"])
@pytest.mark.parametrize("T,E,K,D", SIZES)
def test_combine_and_dispatch_gradient(outer, inner, how, T, E, K, D):
    rng = np.random.default_rng(T * D)
    r, place = routed(T + D + 1, T, E, K)
    ys = put(rng.normal(size=(r.rows, D)), DT[inner], how)
    ys[r.offsets[-1]:] = float("nan")     # rows without a copy are not read
    w = put(rng.random((T, K)), torch.float32, how)
    w[r.place < 0] = float("nan")         # nor are weights of copies without a row
    for weights, wd in ((w, None), (w.bfloat16(), None), (None, 1)):
        buf, out = framed(T, D, DT[outer], how)
        start = rng.normal(size=(T, D))
        for acc in (False, True):
            if acc:
                out.copy_(torch.as_tensor(start))
            old = f64(out) if acc else np.zeros((T, D))
            if weights is None:
                m.muon_moe_dispatch_backward(ys, r, out, accumulate=acc)
            else:
                m.muon_moe_combine(ys, weights, r, out, accumulate=acc)
            want, mass = R.combine(f64(ys), place, None if weights is None else f64(weights))
            want = want + old
            within(f64(out), want, (K + 2) * U * (mass + np.abs(old)) + HALF[outer] * np.abs(want) * (1 + 2.0 ** -7))
            assert untouched(buf, out)


@pytest.mark.parametrize("outer,inner", TYPES)
@pytest.mark.parametrize("how", ["dense", "padded", "shifted"])
@pytest.mark.parametrize("T,E,K,D", SIZES)
def test_combine_gradient(outer, inner, how, T, E, K, D):
    rng = np.random.default_rng(T * D + 5)
    r, place = routed(T + D + 2, T, E, K)
    dout = put(rng.normal(size=(T, D)), DT[outer], how)
    y0 = put(rng.normal(size=(r.rows, D)), DT[inner], how)
    y0[r.offsets[-1]:] = float("nan")
    for wdt in ("f32", "bf16"):
        w = put(rng.random((T, K)), DT[wdt], how)
        w[r.place < 0] = float("nan")
        want, dw_want, mass = R.combine_grad(f64(dout), f64(y0), f64(w), place)
        held = ~np.isnan(want[:, 0])
        for inplace in (False, True):
            bufy, ys = framed(r.rows, D, DT[inner], how)
            ys.copy_(y0)
            buf, dys = framed(r.rows, D, DT[inner], how)
            if inplace:
                buf, dys = bufy, ys
            bufw, dw = framed(T, K, DT[wdt], how)
            m.muon_moe_combine_backward(dout, ys, w, r, dys, dw)
            got = f64(dys)
            within(got[held], want[held], 2 * HALF[inner] * np.abs(want[held]))
            assert np.isnan(got[~held]).all() if inplace else (got[~held] == 7.0).all()
            within(f64(dw), dw_want, (D + 2) * U * mass + HALF[wdt] * np.abs(dw_want) * (1 + 2.0 ** -7))
            assert untouched(buf, dys) and untouched(bufw, dw)
            if not inplace:
                assert torch.equal(torch.nan_to_num(ys), torch.nan_to_num(y0))


@pytest.mark.parametrize("outer,inner", TYPES)
@pytest.mark.parametrize("T,E,K,D", [(4200, 60, 8, 257), (2100, 16, 4, 1111), (1700, 16, 2, 2501),
                                     (330, 9, 3, 8193)])
def test_combine_gradient_of_many_odd_rows(outer, inner, T, E, K, D):
    """Over 16 MB of rows off 16-byte boundaries, which two kernels take one after the other;
    over the rows themselves, too."""
    rng = np.random.default_rng(D)
    r, place = routed(D, T, E, K, drop=0.05)
    assert r.rows * D * 2 > 16e6
    dout = put(rng.normal(size=(T, D)), DT[outer])
    y0 = put(rng.normal(size=(r.rows, D)), DT[inner], "shifted")
    y0[r.offsets[-1]:] = float("nan")
    w = put(rng.random((T, K)), torch.float32)
    want, dw_want, mass = R.combine_grad(f64(dout), f64(y0), f64(w), place)
    held = ~np.isnan(want[:, 0])
    for inplace in (False, True):
        bufy, ys = framed(r.rows, D, DT[inner], "shifted")
        ys.copy_(y0)
        buf, dys = (bufy, ys) if inplace else framed(r.rows, D, DT[inner], "shifted")
        dw = torch.full_like(w, 9.0)
        m.muon_moe_combine_backward(dout, ys, w, r, dys, dw)
        got = f64(dys)
        within(got[held], want[held], 2 * HALF[inner] * np.abs(want[held]))
        assert np.isnan(got[~held]).all() if inplace else (got[~held] == 7.0).all()
        within(f64(dw), dw_want, (D + 3) * U * mass)
        assert untouched(buf, dys)


@pytest.mark.parametrize("outer,inner", TYPES)
@pytest.mark.parametrize("T,E,K", [(50, 8, 2), (21, 16, 6), (9, 30, 17)])
def test_combine_gradient_over_its_own_aligned_rows(outer, inner, T, E, K):
    """Rows on 32-byte boundaries whose last columns fill no 16: dys in the place of ys is
    what it is beside it, bit for bit, and so is the weights' gradient, which needs the
    values that were there."""
    for D in list(range(1, 34)) + [130, 1034, 4111]:
        rng = np.random.default_rng(D + K)
        r, place = routed(D, T, E, K, drop=0.1)
        dout = put(rng.normal(size=(T, D)), DT[outer], "padded")
        w = torch.rand(T, K, device=DEV)
        y0 = rng.normal(size=(r.rows, D))
        bufy, ys = framed(r.rows, D, DT[inner], "padded")
        ys.copy_(torch.as_tensor(y0))
        beside, dw, dw2 = put(y0, DT[inner], "padded"), torch.full_like(w, 9.0), torch.full_like(w, 8.0)
        _, dys = framed(r.rows, D, DT[inner], "padded")
        m.muon_moe_combine_backward(dout, beside, w, r, dys, dw)
        m.muon_moe_combine_backward(dout, ys, w, r, ys, dw2)
        held = torch.as_tensor(place[place >= 0], device=DEV)
        assert torch.equal(dw, dw2) and torch.equal(ys[held], dys[held]) and untouched(bufy, ys)
        _, dw_want, mass = R.combine_grad(f64(dout), f64(beside), f64(w), place)
        within(f64(dw), dw_want, (D + 2) * U * mass)


@pytest.mark.parametrize("wdt", ["f32", "bf16"])
@pytest.mark.parametrize("outer,inner,T,E,K,D", [
    ("f32", "f32", 4100, 60, 8, 129), ("bf16", "f32", 2700, 60, 8, 200), ("f32", "f32", 10300, 8, 2, 200),
    ("f32", "f32", 2100, 60, 8, 255), ("bf16", "bf16", 4000, 60, 8, 256), ("f32", "bf16", 16300, 8, 2, 256),
    ("f32", "bf16", 5500, 16, 6, 256), ("bf16", "bf16", 850, 16, 9, 1111), ("f32", "f32", 500, 32, 17, 515),
    ("f32", "bf16", 620, 32, 17, 801)])
def test_combine_gradient_by_two_kernels(outer, inner, wdt, T, E, K, D):
    """Over 16 MB of rows off 16-byte boundaries: widths of part of a warp in the kernel of the
    weights' gradient, and more choices than that takes at a time.  dys is one product in
    fp32 rounded to the rows' type, to the bit."""
    r, place = routed(D, T, E, K, drop=0.02)
    assert T * K * D * DT[inner].itemsize > 16e6
    g = torch.Generator(device=DEV).manual_seed(D)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    dout = rand(T, D).to(DT[outer])
    y0 = rand(r.rows, D).to(DT[inner])
    w = rand(T, K).to(DT[wdt])
    held = torch.as_tensor(place, device=DEV) >= 0
    at = torch.as_tensor(place, device=DEV)[held]
    rows = (w.float()[:, :, None] * dout.float()[:, None, :])[held].to(DT[inner])
    _, dw_want, mass = R.combine_grad(f64(dout), f64(y0), f64(w), place)
    for inplace in (False, True):
        bufy, ys = framed(r.rows, D, DT[inner], "shifted")
        ys.copy_(y0)
        buf, dys = (bufy, ys) if inplace else framed(r.rows, D, DT[inner], "shifted")
        dw = torch.full_like(w, 9.0)
        m.muon_moe_combine_backward(dout, ys, w, r, dys, dw)
        assert torch.equal(dys[at], rows) and untouched(buf, dys)
        within(f64(dw), dw_want, (D + 3) * U * mass + HALF[wdt] * np.abs(dw_want) * (1 + 2.0 ** -7))


@pytest.mark.parametrize("outer,inner", TYPES)
@pytest.mark.parametrize("wdt", ["f32", "bf16"])
@pytest.mark.parametrize("how", ["dense", "padded", "shifted"])
def test_rows_gradient_is_one_product_rounded_once(outer, inner, wdt, how):
    for T, E, K, D in ((70, 8, 2, 512), (33, 60, 6, 1111), (19, 16, 9, 77), (9, 4, 17, 4100)):
        g = torch.Generator(device=DEV).manual_seed(D)
        r, place = routed(D, T, E, K)
        dout = put(torch.randn(T, D, generator=g, device=DEV), DT[outer], how)
        w = torch.randn(T, K, generator=g, device=DEV).to(DT[wdt])
        ys = put(torch.randn(r.rows, D, generator=g, device=DEV), DT[inner], how)
        _, dys = framed(r.rows, D, DT[inner], how)
        m.muon_moe_combine_backward(dout, ys, w, r, dys, torch.empty_like(w))
        held = torch.as_tensor(place, device=DEV) >= 0
        rows = (w.float()[:, :, None] * dout.float()[:, None, :])[held].to(DT[inner])
        assert torch.equal(dys[torch.as_tensor(place, device=DEV)[held]], rows)


@pytest.mark.parametrize("D", [1, 48, 301, 515])
@pytest.mark.parametrize("outer,inner", TYPES)
def test_no_tokens_and_no_rows(outer, inner, D):
    """Without tokens nothing happens; with tokens but no rows (buffers of none, too) sums and
    weights' gradients are 0, or what was there where it is added to."""
    for T, rows in ((0, 0), (0, 5), (6, 0), (6, 4)):
        E, K = 3, 2
        chosen = torch.full((T, K), -1, device=DEV)
        r = m.Routing.empty(T, K, E, rows=rows)
        ws = m.workspace(m.muon_moe_sort_workspace_size(T, E, K))
        m.muon_moe_sort(chosen, r, ws)
        assert m.muon_get_status(ws) == (m.MUON_OK, 0) and r.offsets.tolist() == [0] * (E + 1)
        x = torch.randn(T, D, device=DEV).to(DT[outer])
        xs = torch.full((rows, D), 7.0, dtype=DT[inner], device=DEV)
        x8 = m.act8_empty(rows, D)
        codes = x8.codes.clone()
        m.muon_moe_dispatch(x, r, xs, x8)
        m.muon_moe_dispatch(x, r, xs)
        assert bool((xs == 7.0).all()) and torch.equal(x8.codes, codes)
        w, out = torch.full((T, K), float("nan"), device=DEV), torch.full_like(x, 9.0)
        for call in (lambda acc: m.muon_moe_combine(xs, w, r, out, accumulate=acc),
                     lambda acc: m.muon_moe_dispatch_backward(xs, r, out, accumulate=acc)):
            out.fill_(9.0)
            call(True)
            assert bool((out == 9.0).all())
            call(False)
            assert bool((out == 0.0).all())
        dw = torch.full_like(w, 9.0)
        m.muon_moe_combine_backward(x, xs, w, r, xs, dw)
        assert bool((xs == 7.0).all()) and bool((dw == 0.0).all())


def test_not_finite_values_reach_their_own_columns_only():
    T, E, K, D = 12, 4, 3, 130
    r, place = routed(3, T, E, K, drop=0.0)
    ys = torch.randn(r.rows, D, device=DEV)
    ys[place[2][0], 17], ys[place[5][1], 129] = float("inf"), float("nan")
    w = torch.rand(T, K, device=DEV)
    out = torch.empty(T, D, device=DEV)
    m.muon_moe_combine(ys, w, r, out)
    bad = torch.zeros(T, D, dtype=torch.bool, device=DEV)
    bad[2, 17] = bad[5, 129] = True
    assert torch.equal(~torch.isfinite(out), bad)
    dout, dys, dw = torch.randn(T, D, device=DEV), torch.empty_like(ys), torch.empty_like(w)
    m.muon_moe_combine_backward(dout, ys, w, r, dys, dw)
    bad = torch.zeros(T, K, dtype=torch.bool, device=DEV)
    bad[2, 0] = bad[5, 1] = True
    assert torch.equal(~torch.isfinite(dw), bad) and bool(torch.isfinite(dys).all())


def test_places_outside_the_rows_are_taken_as_none():
    T, K, D, rows = 6, 2, 40, 7
    r = m.Routing.empty(T, K, 3, rows=rows)
    place = torch.tensor([[0, 6], [7, 1], [-1, 2], [2 ** 31 - 1, 3], [-2 ** 31, 4], [5, 100]], dtype=torch.int32)
    r.place.copy_(place)
    x, xs = torch.randn(T, D, device=DEV), torch.full((rows, D), 7.0, device=DEV)
    m.muon_moe_dispatch(x, r, xs)
    want = R.dispatch(f64(x), place.numpy(), rows)
    assert np.array_equal(f64(xs), want)
    out = torch.empty(T, D, device=DEV)
    m.muon_moe_dispatch_backward(xs, r, out)
    assert torch.equal(out, x * torch.tensor([2., 1, 1, 1, 1, 1], device=DEV)[:, None])
    dys, dw = torch.empty_like(xs), torch.empty(T, K, device=DEV)
    m.muon_moe_combine_backward(x, xs, torch.ones(T, K, device=DEV), r, dys, dw)
    assert torch.equal(dys, xs) and torch.equal((dw != 0).cpu(), (place >= 0) & (place < rows))


def test_row_offsets_past_32_bits():
    """Rows of a buffer of more than 2^32 values; only a few of them are set."""
    T, K, D, rows = 8, 2, 16384, (1 << 18) + 100
    r = m.Routing.empty(T, K, 1, rows=rows)
    at = torch.arange(T * K, dtype=torch.int32).view(T, K)
    r.place.copy_(rows - 1 - 7 * at)
    x = torch.randn(T, D, device=DEV).bfloat16()
    xs = torch.empty(rows, D, dtype=torch.bfloat16, device=DEV)
    x8 = m.act8_empty(rows, D)
    m.muon_moe_dispatch(x, r, xs, x8)
    rowsat = r.place.flatten().long()
    assert torch.equal(xs[rowsat], x.repeat_interleave(K, 0))
    packed = m.act8_empty(T, D)
    m.muon_act8_pack(x, packed)
    assert torch.equal(x8.codes[rowsat], packed.codes.repeat_interleave(K, 0))
    w, out = torch.full((T, K), 0.5, device=DEV), torch.empty_like(x)
    m.muon_moe_combine(xs, w, r, out)
    assert torch.equal(out, x)
    dw = torch.empty(T, K, device=DEV)
    m.muon_moe_combine_backward(x, xs, w, r, xs, dw)
    assert torch.equal(xs[rowsat], (0.5 * x).repeat_interleave(K, 0))


def test_more_items_than_one_launch_takes():
    """Over 2^30 pieces of columns: the tokens are taken in several launches."""
    T = (1 << 29) + 5
    r = m.Routing.empty(T, 1, 2, rows=6)
    r.place.fill_(-1)
    held = torch.tensor([0, 7, (1 << 29) - 1, 1 << 29, (1 << 29) + 3, T - 1], device=DEV)
    r.place[held, 0] = torch.arange(6, dtype=torch.int32, device=DEV)
    x = torch.full((T, 1), 3.0, dtype=torch.bfloat16, device=DEV)
    x[held, 0] = torch.arange(1, 7, device=DEV).bfloat16()
    xs = torch.zeros(6, 1, device=DEV)
    m.muon_moe_dispatch(x, r, xs)
    assert xs[:, 0].tolist() == [1, 2, 3, 4, 5, 6]
    w = torch.full((T, 1), 0.5, dtype=torch.bfloat16, device=DEV)
    dys, dw = torch.zeros_like(xs), torch.full_like(w, 9.0)
    m.muon_moe_combine_backward(x, xs, w, r, dys, dw)
    assert dys[:, 0].tolist() == [0.5, 1, 1.5, 2, 2.5, 3]
    assert dw[held, 0].tolist() == [1, 4, 9, 16, 25, 36] and int((dw != 0).sum()) == 6
    m.muon_moe_combine(xs, w, r, x)
    assert x[held, 0].tolist() == [0.5, 1, 1.5, 2, 2.5, 3] and int((x != 0).sum()) == 6


def test_two_streams_at_once():
    """Two batches on two streams, each with buffers of its own, interleaved call by call."""
    def batch(seed):
        T, E, K, D = 3000 + seed, 20, 4, 515
        chosen = torch.as_tensor(choices(seed, T, E, K, 0.1), device=DEV)
        r = m.Routing.empty(T, K, E)
        ws = m.workspace(m.muon_moe_sort_workspace_size(T, E, K))
        x, w = torch.randn(T, D, device=DEV), torch.rand(T, K, device=DEV)
        xs = torch.zeros(r.rows, D, dtype=torch.bfloat16, device=DEV)
        dys = torch.zeros_like(xs)
        out, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
        calls = [lambda s: m.muon_moe_sort(chosen, r, ws, stream=s),
                 lambda s: m.muon_moe_dispatch(x, r, xs, stream=s),
                 lambda s: m.muon_moe_combine(xs, w, r, out, stream=s),
                 lambda s: m.muon_moe_combine_backward(x, xs, w, r, dys, dw, stream=s),
                 lambda s: m.muon_moe_dispatch_backward(dys, r, dx, stream=s)]
        return calls, (r.offsets, r.place, xs, out, dys, dw, dx)

    both, streams = [batch(1), batch(2)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    alone = []
    for calls, results in both:
        for c in calls:
            c(streams[0])
        torch.cuda.synchronize()
        alone.append([t.clone() for t in results])
        for t in results:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for first, second in zip(both[0][0], both[1][0]):
            first(streams[0])
            second(streams[1])
    torch.cuda.synchronize()
    for (_, results), want in zip(both, alone):
        assert all(torch.equal(a, b) for a, b in zip(results, want))


def test_repeats_its_bits_and_runs_on_another_stream():
    T, E, K, D = 700, 16, 4, 1111
    chosen = torch.as_tensor(choices(2, T, E, K, 0.1), device=DEV)
    x = torch.randn(T, D, device=DEV)
    w, dout = torch.rand(T, K, device=DEV), torch.randn(T, D, device=DEV)

    def once(stream=None):
        r = m.Routing.empty(T, K, E)
        r.order.fill_(-1)
        ws = m.workspace(m.muon_moe_sort_workspace_size(T, E, K))
        xs, dys = (torch.zeros(r.rows, D, device=DEV) for _ in range(2))
        out, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        m.muon_moe_sort(chosen, r, ws, stream=stream)
        m.muon_moe_dispatch(x, r, xs, stream=stream)
        m.muon_moe_combine(xs, w, r, out, stream=stream)
        m.muon_moe_combine_backward(dout, xs, w, r, dys, dw, stream=stream)
        m.muon_moe_dispatch_backward(dys, r, dx, stream=stream)
        torch.cuda.synchronize()
        return [r.offsets, r.order, r.place, xs, out, dys, dw, dx]

    a, b, c = once(), once(), once(torch.cuda.Stream())
    for p, q, s in zip(a, b, c):
        assert torch.equal(p, q) and torch.equal(p, s)


def test_calls_in_a_graph():
    """The whole way captured once and replayed on other choices and values."""
    T, E, K, D = 300, 12, 3, 264
    chosen = torch.as_tensor(choices(1, T, E, K, 0.1), device=DEV)
    x, w, dout = torch.randn(T, D, device=DEV), torch.rand(T, K, device=DEV), torch.randn(T, D, device=DEV)
    r = m.Routing.empty(T, K, E)
    ws = m.workspace(m.muon_moe_sort_workspace_size(T, E, K))
    xs, dys = (torch.zeros(r.rows, D, device=DEV) for _ in range(2))
    out, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)

    def calls():
        m.muon_moe_sort(chosen, r, ws)
        m.muon_moe_dispatch(x, r, xs)
        m.muon_moe_combine(xs, w, r, out)
        m.muon_moe_combine_backward(dout, xs, w, r, dys, dw)
        m.muon_moe_dispatch_backward(dys, r, dx)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for seed in (7, 8):
        c = choices(seed, T, E, K, 0.2)
        chosen.copy_(torch.as_tensor(c))
        x.normal_()
        dout.normal_()
        g.replay()
        torch.cuda.synchronize()
        offsets, order, place, _ = R.sort(c, E)
        assert r.offsets.tolist() == offsets.tolist() and np.array_equal(r.place.cpu().numpy(), place)
        got = [t.clone() for t in (out, dx, dw)]
        calls()
        torch.cuda.synchronize()
        for p, q in zip(got, (out, dx, dw)):
            assert torch.equal(p, q)


def test_two_graphs_share_a_workspace():
    """Two captured sorts (one block, and many) over one workspace, replayed in turn: each
    replay gives what its own inputs give."""
    E, K = 30, 3
    ws = m.workspace(max(m.muon_moe_sort_workspace_size(T, E, K) for T in (100, 9000)))
    work = []
    for T in (100, 9000):
        chosen = torch.as_tensor(choices(T, T, E, K, 0.1), device=DEV)
        r = m.Routing.empty(T, K, E)
        m.muon_moe_sort(chosen, r, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.muon_moe_sort(chosen, r, ws)
        work.append((g, chosen, r))
    for turn in range(4):
        g, chosen, r = work[turn % 2]
        c = choices(50 + turn, chosen.shape[0], E, K, 0.2)
        chosen.copy_(torch.as_tensor(c))
        g.replay()
        torch.cuda.synchronize()
        offsets, order, place, _ = R.sort(c, E)
        assert r.offsets.tolist() == offsets.tolist() and np.array_equal(r.place.cpu().numpy(), place)
        assert np.array_equal(r.order.cpu().numpy()[:len(order)], order)


def test_gradients_against_differences():
    """<d, out(x, w)> with out = combine(f(dispatch(x))), f(v) = v^2: the operators' own
    forward passes at x and w moved by h either way, in fp32 with a large h: the sum is a
    polynomial of degree 2 in x and 1 in w, so central differences are exact, and off by
    roundings alone: 64 U of the sum of the terms' magnitudes over h."""
    T, E, K, D, h = 20, 5, 3, 48, 0.5
    r, place = routed(11, T, E, K)
    x, w, dout = torch.randn(T, D, device=DEV), torch.rand(T, K, device=DEV), torch.randn(T, D, device=DEV)
    dirx, dirw = torch.randn(T, D, device=DEV), torch.randn(T, K, device=DEV)

    def loss(x, w):
        xs, out = torch.zeros(r.rows, D, device=DEV), torch.empty(T, D, device=DEV)
        m.muon_moe_dispatch(x, r, xs)
        m.muon_moe_combine(xs * xs, w, r, out)
        terms = dout.double() * out.double()
        return terms.sum().item(), terms.abs().sum().item()

    xs = torch.zeros(r.rows, D, device=DEV)
    m.muon_moe_dispatch(x, r, xs)
    dys, dw, dx = torch.zeros_like(xs), torch.empty_like(w), torch.empty_like(x)
    m.muon_moe_combine_backward(dout, xs * xs, w, r, dys, dw)
    m.muon_moe_dispatch_backward(2 * xs * dys, r, dx)
    for grad, move in ((dx, lambda s: loss(x + s * dirx, w)), (dw, lambda s: loss(x, w + s * dirw))):
        (up, mu), (down, md) = move(h), move(-h)
        want = (grad.double() * (dirx if grad is dx else dirw).double()).sum().item()
        assert abs((up - down) / (2 * h) - want) <= 64 * U * (mu + md) / h


def test_from_the_choice_to_the_weight_gradient():
    """Sort, dispatch with a checkpoint and the experts' weight gradients together: the
    offsets and the checkpoint go straight into muon_act8_weight_grad."""
    T, E, K, D, F = 500, 6, 2, 96, 64
    chosen = choices(4, T, E, K, 0.1)
    r, _ = run_sort(chosen, E)
    x = torch.randn(T, D, device=DEV)
    xs = torch.zeros(r.rows, D, dtype=torch.bfloat16, device=DEV)
    x8 = m.act8_empty(r.rows, D)
    m.muon_moe_dispatch(x, r, xs, x8)
    dy = torch.randn(r.rows, F, device=DEV).bfloat16()
    G = torch.empty(E, F, D, device=DEV)
    ws = m.workspace(m.muon_act8_weight_grad_workspace_size(r.rows, F, D, E, dy.dtype, G.dtype))
    m.muon_act8_weight_grad(dy, x8, G, ws, offsets=r.offsets)
    assert m.muon_get_status(ws) == (m.MUON_OK, 0)
    one = m.act8_empty(T, D)
    m.muon_act8_pack(x, one)
    xv = torch.empty(T, D, device=DEV)
    m.muon_act8_unpack(one, xv)
    cut, order = r.offsets.tolist(), r.order.long()
    for e in range(E):
        a, b = cut[e], cut[e + 1]
        rows = f64(xv[order[a:b] // K])
        want, mass = f64(dy[a:b]).T @ rows, np.abs(f64(dy[a:b])).T @ np.abs(rows)
        within(f64(G[e]), want, (b - a + 64) * U * mass)


def test_example_layer_gives_back_the_gradient_of_its_input():
    """dx of the example layer against automatic differentiation: 8-bit activations and bf16
    products as in its weights' gradients, 3 % of the norm; and the clipped step is that of
    the gradients times the factor."""
    from tests.test_gpu_example import load
    ex = load()
    layer = ex.MoeLayer(500)
    g = torch.Generator(device=DEV).manual_seed(6)
    x, dy = (torch.randn(500, ex.WIDTH, generator=g, device=DEV) for _ in range(2))
    y = layer.forward(x)
    dx = layer.backward(dy)
    xd = x.double().requires_grad_()
    gate, up, down, router = (t.double() for t in (layer.gate, layer.up, layer.down, layer.router))
    p = (xd @ router.T).softmax(dim=1)
    w = p.gather(1, layer.chosen)
    want = torch.zeros_like(xd)
    for k in range(ex.TOPK):
        for e in range(ex.EXPERTS):
            t = torch.nonzero(layer.chosen[:, k] == e).flatten()
            h = torch.nn.functional.silu(xd[t] @ gate[e].T) * (xd[t] @ up[e].T)
            want = want.index_add(0, t, w[t, k, None] * (h @ down[e].T))
    assert (y - want).norm() <= 0.03 * want.norm()
    f = layer.counts.double() * ex.EXPERTS / (ex.TOPK * 500)
    ((want * dy.double()).sum() + 1e-2 * (f * p.mean(dim=0)).sum()).backward()
    assert (dx - xd.grad).norm() <= 0.03 * xd.grad.norm()
    layer.step(1, max_norm=0.5)
    n, s = R.grad_norm([f64(t) for t in layer.grads.values()], 0.5)
    assert abs(layer.grad_norm.item() - n) <= 7 * U * n and abs(layer.grad_scale.item() - s) <= 9 * U * s
