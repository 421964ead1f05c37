"""Balance loss, 8-bit checkpoints, gated activation and weight gradients on
the GPU against the float64 oracle (oracle/train_ref.py).

Tolerances follow from fp32 arithmetic, U = 2^-24:
  probabilities   an exponential's argument is rounded to U |l - max| and the
                  function adds a few units: relative (16 + |l - max|) 2U.
  logit gradient  the same on each of the two terms f and sum f p, whose own
                  sum has at most 64 roundings: (64 + |l - max|) 2U times
                  coef/N p (f + sum f p).
  loss            all terms positive, fewer than 512 additions in a chain.
  silu            relative (16 + |g|) 2U of each term; in dgate 1 - sigma is
                  known to U absolutely, so its terms are sigma (1 + |g|).
  weight gradient n products added in fp32: (n + 64) U times the sum of their
                  absolute values.
  bf16 outputs    half a unit in the last place (8 significant bits: at most 2^-8
                  relative), on top.
Checkpoints are exact: codes and exponents have to be equal."""
import numpy as np
import pytest
import torch

import newton_schulz_02_gb300 as m
from oracle import train_ref as R
from tests.gpu_util import f64

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


def framed(rows, cols, dtype, how="dense", fill=7.0):
    """(buffer, view): a rows x cols view, dense, with padded rows ("padded"),
    or off every 16-byte boundary ("shifted"), inside a buffer of `fill`."""
    pad = {"dense": 0, "padded": (-cols) % 16 + 16, "shifted": 3}[how]
    lead = 1 if how == "shifted" else 0
    buf = torch.full((max(1, rows * (cols + pad) + lead + 8),), fill, dtype=dtype, device=DEV)
    return buf, buf[lead:].as_strided((rows, cols), (cols + pad, 1))


def put(x, dtype, how="dense"):
    buf, v = framed(*x.shape, dtype, how)
    v.copy_(torch.as_tensor(x, dtype=torch.float32))
    return v


def untouched(buf, view, fill=7.0):
    """Whether everything of the buffer outside the view still holds `fill`."""
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool((buf[keep] == fill).all())


def within(got, want, bound):
    worst = np.max(np.abs(got - want) - bound, initial=-1.0)
    assert not np.isnan(got).any() and worst <= 0.0, f"exceeds its bound by {worst:.3e}"


# ---- balance ----------------------------------------------------------------
def balance_case(seed, T, E, K, S, dtype, padding, how):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, E)) * 2
    if padding and E > K + 1:
        x[:, 1] = -np.inf
    x = put(x, dtype, how)
    xs = f64(x)
    chosen = np.argsort(-xs, axis=1, kind="stable")[:, :K]
    mask = (rng.random(T) > 0.2) if padding else None
    if padding and T:
        chosen[rng.random(T) < 0.1] = -1
    cuts = np.sort(rng.integers(0, T + 1, size=S - 1)) if S > 1 else np.zeros(0, int)
    lo, hi = (min(2, T), max(T - 1, min(2, T))) if padding else (0, T)
    begin = np.concatenate([[lo], np.clip(cuts, lo, hi), [hi]])
    return x, xs, chosen, begin, mask


def run_balance(x, chosen, begin, mask, score, coef, idx=torch.int64, dl=None, dloss=None, acc=False):
    T, E = x.shape
    S = 1 if begin is None else len(begin) - 1
    dev = lambda a, dt: None if a is None else torch.as_tensor(np.ascontiguousarray(a)).to(DEV, dt)
    b = m.Balance(x, dev(chosen, idx), dev(begin, torch.int32), dev(mask, torch.bool), score, coef)
    loss = torch.full((1,), 5.0, device=DEV)
    counts = torch.full((E,), 99, dtype=torch.int32, device=DEV)
    load = torch.full((S, E), 5.0, device=DEV)
    ws = m.workspace(m.muon_balance_workspace_size(T, E, S))
    ws.fill_(255)
    if dl is None:
        dl = torch.full((T, E), 5.0, dtype=x.dtype, device=DEV)
    m.muon_balance_forward(b, loss, counts, load, ws)
    m.muon_balance_backward(b, load, dl, dloss=dloss, accumulate=acc)
    code, flags = m.muon_get_status(ws)
    assert code == m.MUON_OK
    return loss, counts, load, dl, flags


def grad_bound(ref, xs, half):
    top = np.max(np.where(np.isinf(xs), -1e30, xs), axis=1, keepdims=True, initial=-1e30)
    gap = np.minimum(np.abs(xs - top), 200.0)
    return ref["mass"] * ((64 + gap) * 2 * U + half) + 1e-37


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,K,S,padding,how", [
    (1, 1, 1, 1, False, "dense"), (1, 8, 2, 1, False, "dense"), (0, 8, 2, 2, False, "dense"),
    (33, 8, 2, 3, True, "shifted"), (257, 31, 3, 5, True, "dense"), (100, 64, 6, 1, False, "padded"),
    (1000, 60, 6, 40, True, "dense"), (77, 100, 8, 7, True, "shifted"), (3000, 128, 4, 9, False, "dense"),
    (700, 256, 8, 300, True, "padded"), (65, 257, 2, 1, True, "dense"), (90, 512, 8, 4, False, "shifted"),
    (41, 1024, 8, 2, True, "dense"), (70001, 16, 2, 3, True, "dense")])
def test_balance(score, dtype, T, E, K, S, padding, how):
    x, xs, chosen, begin, mask = balance_case(T + E, T, E, K, S, DT[dtype], padding, how)
    buf, dl = framed(T, E, DT[dtype], how)
    loss, counts, load, dl, flags = run_balance(x, chosen, begin, mask, score, 0.25, dl=dl)
    ref = R.balance(xs, chosen, begin, mask, score, np.float32(0.25))
    assert flags == 0 and counts.cpu().numpy().tolist() == ref["counts"].tolist()
    assert abs(loss.item() - ref["loss"]) <= 512 * U * ref["loss"] + 1e-30
    within(f64(load), ref["load"], 8 * U * ref["load"])
    within(f64(dl), ref["grad"], grad_bound(ref, xs, HALF[dtype]))
    assert untouched(buf, dl)


@pytest.mark.parametrize("T,E,S", [(9000, 20, 5000), (300, 40, 6000), (40000, 8, 64)])
def test_balance_many_sequences(T, E, S):
    """Thousands of sequences, most of one token or none; bounds out of order
    are flagged there too."""
    x, xs, chosen, begin, mask = balance_case(T, T, E, 3, S, torch.float32, True, "dense")
    loss, counts, load, dl, flags = run_balance(x, chosen, begin, mask, "softmax", 0.25)
    ref = R.balance(xs, chosen, begin, mask, "softmax", np.float32(0.25))
    assert flags == 0 and counts.cpu().numpy().tolist() == ref["counts"].tolist()
    assert abs(loss.item() - ref["loss"]) <= 512 * U * ref["loss"] + 1e-30
    within(f64(load), ref["load"], 8 * U * ref["load"])
    within(f64(dl), ref["grad"], grad_bound(ref, xs, U))
    begin[S // 2] = T + 7
    assert run_balance(x, chosen, begin, mask, "softmax", 0.25)[4] == m.MUON_FLAG_INDEX


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K,off", [(352, 4, 2, 2), (1000, 8, 6, 2), (64, 8, 8, 0), (300, 33, 31, 2)])
def test_balance_every_enabled_expert_taken(score, T, E, K, off):
    """Tokens that take all experts with a probability: they cannot change the
    loss, and the gradient is 0, not what is left of a difference."""
    x = torch.randn(T, E, device=DEV) * 3
    if off:
        x[:, 1] = x[:, E - 1] = float("-inf")
    chosen = torch.topk(x, K).indices.cpu().numpy()
    loss, counts, load, dl, flags = run_balance(x, chosen, [0, T // 3, T], None, score, 1.0)
    assert flags == 0 and not dl.any()
    ref = R.balance(f64(x), chosen, [0, T // 3, T], None, score, 1.0)
    assert abs(loss.item() - ref["loss"]) <= 512 * U * ref["loss"]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K,on", [(300, 64, 8, 8), (300, 128, 8, 8), (500, 256, 8, 8), (77, 40, 1, 1), (60, 64, 16, 16),
                                      (200, 257, 3, 3), (90, 512, 300, 300), (41, 1024, 2, 2), (50, 33, 9, 9)])
def test_balance_every_enabled_expert_taken_among_disabled_ones(score, T, E, K, on):
    """The same routing among many disabled experts: 0 where the header says so,
    else what rounding leaves of two equal terms; a sequence beside it that does
    choose has its gradient."""
    g = torch.Generator(device=DEV).manual_seed(T + E)
    x = torch.full((T, E), float("-inf"), device=DEV)
    cols = torch.randperm(E, generator=g, device=DEV)[:on]
    x[:, cols] = torch.randn(T, on, generator=g, device=DEV) * 3
    half = T // 2
    for rest in (x[half:], torch.randn(T - half, E, generator=g, device=DEV) * 3):
        x[half:] = rest
        chosen = torch.topk(x, K).indices.cpu().numpy()
        loss, counts, load, dl, flags = run_balance(x, chosen, [0, half, T], None, score, 1.0)
        ref = R.balance(f64(x), chosen, [0, half, T], None, score, 1.0)
        assert flags == 0
        within(f64(dl), ref["grad"], grad_bound(ref, f64(x), U))
        assert np.all(np.abs(f64(dl[:half])) <= 2.0 ** -17 * ref["mass"][:half])
        if E <= 64 and 4 * K >= E:
            assert not dl[:half].any()


def test_balance_one_sequence_without_bounds_equals_with():
    x, xs, chosen, _, _ = balance_case(3, 500, 48, 4, 1, torch.float32, False, "dense")
    a = run_balance(x, chosen, None, None, "softmax", 0.1)
    b = run_balance(x, chosen, [0, 500], None, "softmax", 0.1, idx=torch.int32)
    for p, q in zip(a[:4], b[:4]):
        assert torch.equal(p, q)


def test_balance_masked_tokens_are_not_read():
    """NaN and infinities in padding, outside the sequences, and as disabled experts."""
    T, E, K = 300, 24, 3
    x, xs, chosen, begin, mask = balance_case(9, T, E, K, 4, torch.float32, True, "dense")
    clean = run_balance(x, chosen, begin, mask, "softmax", 0.1)
    dirty = x.clone()
    off = torch.as_tensor(~mask)
    off[: begin[0]] = True
    off[begin[-1]:] = True
    dirty[off.to(DEV)] = float("nan")
    dirty[int(torch.nonzero(off)[0])] = float("inf")
    got = run_balance(dirty, chosen, begin, mask, "softmax", 0.1)
    for p, q in zip(clean[:4], got[:4]):
        assert torch.equal(p, q)
    assert not got[3][off.to(DEV)].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_rows_without_an_expert(score):
    """Rows of -inf alone have no probability and no gradient; rows of the
    type's lowest value are uniform under softmax."""
    x = torch.randn(40, 10, device=DEV)
    x[3] = float("-inf")
    x[5] = torch.finfo(torch.float32).min
    chosen = torch.topk(x, 2).indices.cpu().numpy()
    xs = f64(x)
    loss, counts, load, dl, flags = run_balance(x, chosen, None, None, score, 1.0)
    with np.errstate(over="ignore"):
        ref = R.balance(xs, chosen, None, None, score, 1.0)
    assert abs(loss.item() - ref["loss"]) <= 512 * U * ref["loss"]
    assert not dl[3].any()
    within(f64(dl), ref["grad"], grad_bound(ref, xs, U))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,K", [(10, 2), (60, 6), (200, 8), (256, 8), (600, 4)])
def test_balance_sigmoid_rows_far_below_zero(E, K, dtype):
    """sigma / sum sigma of rows whose logits are all so low that fp32 has no sigmoid
    for them, beside ordinary rows, with disabled experts, in place and added."""
    g = torch.Generator(device=DEV).manual_seed(E)
    x = torch.randn(120, E, generator=g, device=DEV) * 2
    for r, shift in ((3, -25.0), (7, -60.0), (8, -90.0), (31, -150.0), (64, -500.0), (65, -690.0), (100, -100.0)):
        x[r] += shift
    x[8, 1::2] = float("-inf")
    x[9] = float("-inf")
    x[100, 0] = 5.0            # one ordinary logit among low ones
    x = x.to(DT[dtype])
    chosen = torch.topk(x.float(), K).indices.cpu().numpy()
    loss, counts, load, dl, flags = run_balance(x, chosen, [0, 50, 120], None, "sigmoid", 1.0)
    ref = R.balance(f64(x), chosen, [0, 50, 120], None, "sigmoid", 1.0)
    assert flags == 0 and abs(loss.item() - ref["loss"]) <= 512 * U * ref["loss"]
    within(f64(dl), ref["grad"], grad_bound(ref, f64(x), HALF[dtype]))
    assert (dl[[7, 8, 31, 64, 65]] != 0).any(dim=1).all() and not dl[9].any()
    mine = x.clone()
    assert torch.equal(run_balance(mine, chosen, [0, 50, 120], None, "sigmoid", 1.0, dl=mine)[3], dl)
    start = torch.randn(120, E, generator=g, device=DEV)
    got = run_balance(x, chosen, [0, 50, 120], None, "sigmoid", 1.0, dl=start.clone(), acc=True)[3]
    total = f64(start) + ref["grad"]
    within(f64(got), total, grad_bound(ref, f64(x), U) + U * np.abs(total) * 1.01)


def test_balance_nan_propagates_and_bad_indices_are_flagged():
    x = torch.randn(64, 16, device=DEV)
    chosen = torch.topk(x, 2).indices.cpu().numpy()
    bad = chosen.copy()
    bad[7, 1], bad[9, 0] = 16, -2
    a = run_balance(x, chosen, None, None, "softmax", 1.0)
    b = run_balance(x, bad, None, None, "softmax", 1.0)
    assert a[4] == 0 and b[4] == m.MUON_FLAG_INDEX and b[1].sum().item() == 126
    assert run_balance(x, chosen, [0, 70], None, "softmax", 1.0)[4] == m.MUON_FLAG_INDEX
    assert run_balance(x, chosen, [0, 40, 20, 64], None, "softmax", 1.0)[4] == m.MUON_FLAG_INDEX
    x[5, 3] = float("nan")
    n = run_balance(x, chosen, None, None, "softmax", 1.0)
    assert torch.isnan(n[0]).all() and torch.isnan(n[3][5]).all() and not torch.isnan(n[3][6]).any()


@pytest.mark.parametrize("begin", [[0, 64, 0, 64], [0, 40, 20, 64], [64, 0], [0, 200, -3, 64, 10], [50, 10, 64, 0]])
def test_balance_bounds_out_of_order_do_not_read_the_workspace(begin):
    """What the workspace held before shows in no output, whatever the bounds."""
    x = torch.randn(64, 16, device=DEV)
    b = m.Balance(x, torch.topk(x, 2).indices, torch.tensor(begin, dtype=torch.int32, device=DEV))
    seqs, first = len(begin) - 1, None
    for fill in (0, 1, 255):
        loss, counts = torch.empty(1, device=DEV), torch.empty(16, dtype=torch.int32, device=DEV)
        load, dl = torch.empty(seqs, 16, device=DEV), torch.empty(64, 16, device=DEV)
        ws = m.workspace(m.muon_balance_workspace_size(64, 16, seqs))
        ws.fill_(fill)
        m.muon_balance_forward(b, loss, counts, load, ws)
        m.muon_balance_backward(b, load, dl)
        assert m.muon_get_status(ws) == (m.MUON_OK, m.MUON_FLAG_INDEX)
        got = [loss, counts, load, dl]
        first = first or got
        assert all(torch.isfinite(t).all() and torch.equal(t, f) for t, f in zip(got, first))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_balance_accumulate_scale_and_in_place(dtype):
    x, xs, chosen, begin, mask = balance_case(4, 210, 40, 4, 3, DT[dtype], True, "dense")
    ref = R.balance(xs, chosen, begin, mask, "softmax", np.float32(0.5))
    start = torch.randn(210, 40, device=DEV).to(DT[dtype])
    dl = start.clone()
    scale = torch.tensor([3.0], device=DEV)
    run_balance(x, chosen, begin, mask, "softmax", 0.5, dl=dl, dloss=scale, acc=True)
    want = f64(start) + 3 * ref["grad"]
    within(f64(dl), want, 3 * grad_bound(ref, xs, U) + HALF[dtype] * np.abs(want) * 1.01 + 1e-37)
    skipped = ref["mass"].sum(axis=1) == 0
    assert torch.equal(dl[skipped], start[skipped])
    fresh = run_balance(x, chosen, begin, mask, "softmax", 0.5)[3]
    inplace = x.clone()
    got = run_balance(inplace, chosen, begin, mask, "softmax", 0.5, dl=inplace)[3]
    assert torch.equal(got, fresh)


def test_balance_repeats_its_bits():
    x, xs, chosen, begin, mask = balance_case(8, 20000, 96, 6, 12, torch.bfloat16, True, "dense")
    a = run_balance(x, chosen, begin, mask, "softmax", 0.5)
    for _ in range(3):
        b = run_balance(x, chosen, begin, mask, "softmax", 0.5)
        for p, q in zip(a[:4], b[:4]):
            assert torch.equal(p, q)


def test_balance_gradient_against_differences():
    """Directional differences of the GPU's own loss: a step of 2^-6 leaves a
    truncation of its square and a rounding of 512 U / step of the loss."""
    x, xs, chosen, begin, mask = balance_case(2, 64, 12, 2, 3, torch.float32, False, "dense")
    rng = np.random.default_rng(0)
    g = f64(run_balance(x, chosen, begin, mask, "softmax", 1.0)[3])
    for _ in range(4):
        v = torch.as_tensor(rng.normal(size=(64, 12)), dtype=torch.float32, device=DEV)
        h = 2.0 ** -6
        up, dn = (run_balance(x + s * h * v, chosen, begin, mask, "softmax", 1.0)[0].item()
                  for s in (1, -1))
        num = (up - dn) / (2 * h)
        size = np.abs(g * f64(v)).sum()
        assert abs(num - (g * f64(v)).sum()) <= 20 * h * h * size + 512 * U * 4 / h


# ---- checkpoints ------------------------------------------------------------
def mixed(rng, rows, cols):
    """Rows of very different sizes, outliers, zeros, ties and tiny values."""
    x = rng.normal(size=(rows, cols)) * np.exp2(rng.integers(-30, 30, size=(rows, 1)))
    x[rng.random((rows, cols)) < 0.05] *= 64
    x[rng.random((rows, cols)) < 0.1] = 0.0
    if rows > 3:
        x[0] = 0.0
        x[1] = np.round(x[1] / np.max(np.abs(x[1]) + 1e-300) * 254) / 2     # ties
        x[2] *= 2.0 ** -120
        x[3, 0] = 2.0 ** -149
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("how", ["dense", "padded", "shifted"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (5, 31), (7, 33), (64, 64), (3, 1000),
                                       (130, 1111), (17, 4096), (0, 40)])
def test_act8_round_trip(dtype, how, rows, cols):
    x = put(mixed(np.random.default_rng(rows * 7 + cols), rows, cols), DT[dtype], how)
    a = m.act8_empty(rows, cols)
    a.codes.fill_(55)
    a.exps.fill_(77)
    m.muon_act8_pack(x, a)
    codes, exps = R.act8_encode(f64(x))
    nb = exps.shape[1]
    assert np.array_equal(a.codes.cpu().numpy(), codes)
    assert np.array_equal(a.exps.cpu().numpy()[:, :nb], exps)
    assert (a.exps[:, nb:] == 77).all()
    for out_dtype in (torch.float32, torch.bfloat16):
        buf, back = framed(rows, cols, out_dtype, how)
        m.muon_act8_unpack(a, back)
        assert np.array_equal(f64(back), R.act8_decode(codes, exps, cols))
        assert untouched(buf, back)


def test_act8_not_finite_and_extreme():
    big = torch.finfo(torch.float32).max
    x = torch.zeros(4, 96, device=DEV)
    x[0, 3], x[0, 40], x[1, 95] = float("nan"), float("inf"), float("-inf")
    x[2, 0], x[2, 1], x[3, 64] = big, -big, 1e-45
    for view in (x, torch.cat([x, x[:, :1]], 1)[:, :96], torch.cat([x, x], 1)[:, 1:97]):
        a = m.act8_empty(4, 96)
        m.muon_act8_pack(view, a)
        back = torch.empty(4, 96, device=DEV)
        m.muon_act8_unpack(a, back)
        codes, exps = R.act8_encode(f64(view))
        assert np.array_equal(a.exps.cpu().numpy()[:, :3], exps)
        assert np.array_equal(f64(back), R.act8_decode(codes, exps, 96), equal_nan=True)
        assert not torch.isinf(back).any()


def test_act8_one_row_of_many():
    """Single rows of a checkpoint as checkpoints of their own, in every pass."""
    rows, cols = 6, 200
    x = torch.randn(rows, cols, device=DEV)
    codes = torch.full((rows, 256), 55, dtype=torch.int8, device=DEV)
    exps = torch.full((rows, 16), 77, dtype=torch.uint8, device=DEV)
    for r in range(rows):
        m.muon_act8_pack(x[r:r + 1], m.Act8(codes[r:r + 1, :224], exps[r:r + 1, :7], cols))
    want, we = R.act8_encode(f64(x))
    assert np.array_equal(codes[:, :224].cpu().numpy(), want) and (codes[:, 224:] == 55).all()
    assert np.array_equal(exps[:, :7].cpu().numpy(), we) and (exps[:, 7:] == 77).all()
    back = torch.empty(1, cols, device=DEV)
    one = m.Act8(codes[4:5, :224], exps[4:5, :7], cols)
    m.muon_act8_unpack(one, back)
    assert np.array_equal(f64(back), R.act8_decode(want[4:5], we[4:5], cols))
    dy, G = torch.randn(1, 40, device=DEV), torch.empty(1, 40, cols, device=DEV)
    assert run_wgrad(dy, one, G, torch.tensor([0, 1], dtype=torch.int32, device=DEV)) == 0
    full, size = R.weight_grads(f64(dy), f64(back), [0, 1])
    within(f64(G), full, wgrad_bound(size, full, [0, 1], U))


def test_act8_offsets_past_32_bits():
    """70000 rows of 32768 columns: elements past 2^31 in the source and the codes."""
    rows, cols = 70000, 32768
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    some = torch.tensor([0, 1, 65535, 65536, 69998, 69999], device=DEV)
    x[some] = torch.randn(6, cols, generator=g, device=DEV).bfloat16()
    a = m.act8_empty(rows, cols)
    m.muon_act8_pack(x, a)
    codes, exps = R.act8_encode(f64(x[some][:, -512:]))
    assert np.array_equal(a.codes[some][:, -512:].cpu().numpy(), codes)
    back = torch.full_like(x, 3.0)
    m.muon_act8_unpack(a, back)
    assert np.array_equal(f64(back[some][:, -512:]), R.act8_decode(codes, exps, 512))
    assert int((back != 0).sum(dtype=torch.int64)) <= 6 * cols


# ---- gated activation -------------------------------------------------------
def swiglu_bounds(d, g, u, half):
    s = R.sigmoid(g)
    rel = (16 + np.abs(g)) * 2 * U
    h, (dg, du) = R.swiglu(g, u), R.swiglu_grad(d, g, u)
    tiny = 1e-35 * (1 + np.abs(d)) * (1 + np.abs(u)) * (1 + np.abs(g))
    return (np.abs(h) * (rel + half) + tiny,
            np.abs(d * u) * s * (1 + np.abs(g)) * rel + np.abs(dg) * half + tiny,
            np.abs(du) * (rel + half) + tiny)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("how", ["dense", "padded", "shifted"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 32), (19, 1531), (40, 256), (0, 16), (9, 2049)])
def test_swiglu(dtype, how, rows, cols):
    rng = np.random.default_rng(rows + cols)
    gate, up, dh = (put(rng.normal(size=(rows, cols)) * s, DT[dtype], how) for s in (4.0, 2.0, 1e-2))
    if rows > 2:
        gate[0, :3] = torch.tensor([100.0, -100.0, 0.0], dtype=DT[dtype], device=DEV)[: min(3, cols)]
    g8, u8, h8 = (m.act8_empty(rows, cols) for _ in range(3))
    (hb, h), (gb, dgate), (ub, dup) = (framed(rows, cols, DT[dtype], how) for _ in range(3))
    m.muon_act8_swiglu_forward(gate, up, h, g8, u8)
    m.muon_act8_swiglu_backward(dh, g8, u8, dgate, dup, h8)
    for kept, t in ((g8, gate), (u8, up)):
        codes, exps = R.act8_encode(f64(t))
        assert np.array_equal(kept.codes.cpu().numpy(), codes)
        assert np.array_equal(kept.exps.cpu().numpy()[:, : exps.shape[1]], exps)
    within(f64(h), R.swiglu(f64(gate), f64(up)),
           swiglu_bounds(f64(dh), f64(gate), f64(up), HALF[dtype])[0])
    g, u = (R.act8_decode(*R.act8_encode(f64(t)), cols) for t in (gate, up))
    bounds = swiglu_bounds(f64(dh), g, u, HALF[dtype])
    dg, du = R.swiglu_grad(f64(dh), g, u)
    within(f64(dgate), dg, bounds[1])
    within(f64(dup), du, bounds[2])
    # h8: within half a step of the recomputed h, itself within its own bound
    hv = R.swiglu(g, u)
    step = np.repeat(np.ldexp(1.0, h8.exps.cpu().numpy().astype(int)[:, : -(-cols // 32)] - 127), 32,
                     axis=1)[:, :cols]
    back = torch.empty(rows, cols, device=DEV)
    m.muon_act8_unpack(h8, back)
    within(f64(back), hv, step / 2 + swiglu_bounds(f64(dh), g, u, U)[0])
    if cols % 32:
        assert not h8.codes[:, cols:].any()
    for b, v in ((hb, h), (gb, dgate), (ub, dup)):
        assert untouched(b, v)
    # without h8, and with dgate in dh's place: the same bits
    again, dh2 = torch.empty_like(dup), dh.clone() if how == "dense" else dh
    m.muon_act8_swiglu_backward(dh2, g8, u8, dh2, again)
    assert torch.equal(dh2, dgate) and torch.equal(again, dup)


def test_swiglu_gradient_against_differences():
    """Differences of the GPU's h in fp32 at the checkpoint's own values."""
    rng = np.random.default_rng(6)
    g8, u8 = m.act8_empty(8, 96), m.act8_empty(8, 96)
    t = lambda s: torch.as_tensor(rng.normal(size=(8, 96)) * s, dtype=torch.float32, device=DEV)
    gate, up, dh = t(2.0), t(1.0), t(1.0)
    m.muon_act8_pack(gate, g8)
    m.muon_act8_pack(up, u8)
    g, u = torch.empty_like(gate), torch.empty_like(up)
    m.muon_act8_unpack(g8, g)
    m.muon_act8_unpack(u8, u)
    dgate, dup = torch.empty_like(g), torch.empty_like(g)
    m.muon_act8_swiglu_backward(dh, g8, u8, dgate, dup)
    spare = [m.act8_empty(8, 96) for _ in range(2)]

    def h(a, b):
        out = torch.empty_like(a)
        m.muon_act8_swiglu_forward(a, b, out, *spare)
        return f64(out)

    e = 2.0 ** -7
    # truncation e^2/6 of a third derivative below 1, roundings 32 U (1 + |h|) / e
    tol = lambda w: np.abs(f64(dh)) * (np.abs(w) + 1) * (e * e + 64 * U * 20 / e)
    within(f64(dgate), f64(dh) * (h(g + e, u) - h(g - e, u)) / (2 * e), tol(f64(u)))
    within(f64(dup), f64(dh) * (h(g, u + e) - h(g, u - e)) / (2 * e), tol(f64(g)))


# ---- weight gradients -------------------------------------------------------
def wgrad_case(seed, offsets, rows, out, inp, dy, how):
    rng = np.random.default_rng(seed)
    d = put(rng.normal(size=(rows, out)) * np.exp2(rng.integers(-8, 3, size=(rows, 1))), DT[dy], how)
    x8 = m.act8_empty(rows, inp)
    x8.codes.fill_(-128)    # what lies between cols and the row's end must not matter
    x8.exps.fill_(255)
    x = put(mixed(rng, rows, inp) if rows < 4 else rng.normal(size=(rows, inp)) * 3, DT["f32"])
    m.muon_act8_pack(x, x8)
    xs = R.act8_decode(*R.act8_encode(f64(x)), inp) if rows * inp < 40000 else None
    if xs is None:
        back = torch.empty(rows, inp, device=DEV)
        m.muon_act8_unpack(x8, back)
        xs = f64(back)
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)
    return d, x8, off, f64(d), xs


def run_wgrad(d, x8, G, off, acc=False, stream=None):
    n_exp = 1 if G.dim() == 2 else G.shape[0]
    ws = m.workspace(m.muon_act8_weight_grad_workspace_size(
        x8.shape[0], d.shape[1], x8.shape[1], n_exp, d.dtype, G.dtype))
    ws.fill_(255)
    m.muon_act8_weight_grad(d, x8, G, ws, offsets=off, accumulate=acc, stream=stream)
    code, flags = m.muon_get_status(ws, stream) if stream is not None else m.muon_get_status(ws)
    assert code == m.MUON_OK
    return flags


def wgrad_bound(size, want, offsets, half):
    n = np.diff(offsets)[:, None, None]
    return (n + 64) * U * size + half * np.abs(want) * 1.01 + 1e-37


SPANS = [
    ([0, 0], 0, 40, 24), ([0, 1], 1, 8, 8), ([0, 1], 1, 1, 1), ([0, 5], 5, 33, 7),
    ([0, 64], 64, 256, 128), ([0, 63, 63, 200], 200, 128, 256), ([0, 7, 8, 8, 80, 81], 90, 72, 200),
    ([3, 20, 300], 310, 300, 520), ([0, 1000], 1000, 136, 264), ([0, 129, 257, 640], 640, 512, 256),
    ([0, 17, 17, 17, 40, 41, 61, 61, 61], 61, 520, 264), ([0, 3000], 3000, 24, 1000),
    ([0, 4097], 4097, 256, 512), ([0, 500, 900], 900, 1111, 333)]


@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("dy", ["bf16", "f32"])
@pytest.mark.parametrize("offsets,rows,out,inp", SPANS)
def test_weight_grad(offsets, rows, out, inp, dy, grad):
    d, x8, off, ds, xs = wgrad_case(rows + out, offsets, rows, out, inp, dy, "dense")
    E = len(offsets) - 1
    G = torch.full((E, out, inp), 3.0, dtype=DT[grad], device=DEV)
    assert run_wgrad(d, x8, G, off) == 0
    want, size = R.weight_grads(ds, xs, offsets)
    within(f64(G), want, wgrad_bound(size, want, offsets, HALF[grad]))
    start = torch.randn(E, out, inp, device=DEV).to(DT[grad])
    G = start.clone()
    run_wgrad(d, x8, G, off, acc=True)
    total = f64(start) + want
    within(f64(G), total, wgrad_bound(size, total, offsets, HALF[grad]) + U * np.abs(total))


@pytest.mark.parametrize("how", ["padded", "shifted"])
@pytest.mark.parametrize("dy", ["bf16", "f32"])
@pytest.mark.parametrize("offsets,rows,out,inp", [SPANS[6], SPANS[7], SPANS[10], SPANS[13]])
def test_weight_grad_strides(offsets, rows, out, inp, dy, how):
    """Rows of dy and of G with gaps, and off every 16-byte boundary; G as
    separate matrices of a Group in reversed order."""
    d, x8, off, ds, xs = wgrad_case(rows, offsets, rows, out, inp, dy, how)
    E = len(offsets) - 1
    want, size = R.weight_grads(ds, xs, offsets)
    bound = wgrad_bound(size, want, offsets, HALF["f32"])
    pad = 24 if how == "padded" else 3
    lead = 0 if how == "padded" else 1
    buf = torch.full((E * out * (inp + pad) + lead,), 7.0, device=DEV)
    G = buf[lead:].as_strided((E, out, inp), (out * (inp + pad), inp + pad, 1))
    assert run_wgrad(d, x8, G, off) == 0
    within(f64(G), want, bound)
    assert untouched(buf, G)
    if how == "padded" and inp % 8 == 0:
        mats = [G[e] for e in reversed(range(E))]
        buf.fill_(7.0)
        grp = m.Group(mats, mats, mats)
        ws = m.workspace(m.muon_act8_weight_grad_workspace_size(rows, out, inp, E, d.dtype, G.dtype))
        m.muon_act8_weight_grad(d, x8, grp, ws, offsets=off)
        within(f64(G)[::-1], want, bound)
        assert untouched(buf, G)


@pytest.mark.parametrize("dy", ["bf16", "f32"])
def test_weight_grad_other_experts_rows_do_not_leak(dy):
    """NaN and infinities in another expert's tokens (dy and checkpoint), right
    up to the span's ends, and in rows that no expert owns."""
    offsets, rows, out, inp = [5, 38, 100, 171], 180, 136, 160
    d, x8, off, ds, xs = wgrad_case(1, offsets, rows, out, inp, dy, "dense")
    want, size = R.weight_grads(ds, xs, offsets)
    for sl in (slice(0, 5), slice(38, 100), slice(171, 180)):
        d[sl] = float("nan")
        d[sl.start] = float("inf")
        x8.exps[sl] = 255
    G = torch.full((3, out, inp), 3.0, device=DEV)
    run_wgrad(d, x8, G, off)
    bound = wgrad_bound(size, want, offsets, U)
    for e in (0, 2):
        within(f64(G[e]), want[e], bound[e])
    assert torch.isnan(G[1]).all()


@pytest.mark.parametrize("dy", ["bf16", "f32"])
def test_weight_grad_both_ctas_operands_arrive(dy):
    """Many short spans side by side with experts of NaN, on all pairs at once and
    again and again: each CTA of a pair zeroes its own half of the neighbours' rows
    and the pair's products read both."""
    rng = np.random.default_rng(12)
    offsets = np.concatenate([[0], np.cumsum(rng.integers(1, 130, size=64))]).tolist()
    rows, out, inp = offsets[-1], 512, 512
    d, x8, off, ds, xs = wgrad_case(12, offsets, rows, out, inp, dy, "dense")
    want, size = R.weight_grads(ds, xs, offsets)
    bound = wgrad_bound(size, want, offsets, U)
    for e in range(1, 64, 2):
        d[offsets[e]:offsets[e + 1]] = float("nan")
        x8.exps[offsets[e]:offsets[e + 1]] = 255
    first = torch.empty(64, out, inp, device=DEV)
    assert run_wgrad(d, x8, first, off) == 0
    within(f64(first[::2]), want[::2], bound[::2])
    assert torch.isnan(first[1::2]).all()
    for _ in range(20):
        G = torch.full_like(first, 3.0)
        assert run_wgrad(d, x8, G, off) == 0
        assert torch.equal(G[::2], first[::2])


@pytest.mark.parametrize("dy", ["bf16", "f32"])
def test_weight_grad_nan_block_reaches_its_columns_only(dy):
    offsets, rows, out, inp = [0, 70], 70, 64, 160
    d, x8, off, ds, xs = wgrad_case(2, offsets, rows, out, inp, dy, "dense")
    x8.exps[33, 2] = 255
    G = torch.empty(out, inp, device=DEV)
    run_wgrad(d, x8, G, off)
    bad = torch.isnan(G)
    assert bad[:, 64:96].all() and not bad[:, :64].any() and not bad[:, 96:].any()


def test_weight_grad_bad_offsets_are_cut_and_flagged():
    d, x8, off, ds, xs = wgrad_case(3, [0, 50], 50, 40, 64, "bf16", "dense")
    G = torch.empty(2, 40, 64, device=DEV)
    bad = torch.tensor([-5, 30, 60], dtype=torch.int32, device=DEV)
    assert run_wgrad(d, x8, G, bad) == m.MUON_FLAG_INDEX
    want, size = R.weight_grads(ds, xs, [0, 30, 50])
    within(f64(G), want, wgrad_bound(size, want, [0, 30, 50], U))
    down = torch.tensor([0, 30, 20], dtype=torch.int32, device=DEV)
    assert run_wgrad(d, x8, G, down) == m.MUON_FLAG_INDEX
    assert not G[1].any()


def test_weight_grad_repeats_its_bits_and_runs_on_another_stream():
    offsets, rows, out, inp = [0, 800, 801, 2500], 2500, 300, 640
    d, x8, off, ds, xs = wgrad_case(4, offsets, rows, out, inp, "bf16", "dense")
    first = torch.empty(3, out, inp, device=DEV)
    run_wgrad(d, x8, first, off)
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream()):
        G = torch.full_like(first, 2.0)
        torch.cuda.synchronize()
        run_wgrad(d, x8, G, off, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(G, first)


def test_weight_grad_row_offsets_past_32_bits():
    """dy rows 2^23 elements apart: 300 of them span 5 GB."""
    rows, out, inp, gap = 300, 64, 96, 1 << 23
    buf = torch.zeros(rows * gap, dtype=torch.bfloat16, device=DEV)
    d = buf.as_strided((rows, out), (gap, 1))
    src, x8, off, ds, xs = wgrad_case(5, [0, rows], rows, out, inp, "bf16", "dense")
    d.copy_(src)
    G = torch.empty(1, out, inp, device=DEV)
    run_wgrad(d, x8, G, off)
    want, size = R.weight_grads(ds, xs, [0, rows])
    within(f64(G), want, wgrad_bound(size, want, [0, rows], U))


def test_weight_grad_against_differences():
    """G . V equals the change of sum_t dy_t . (W x_t) along V (it is linear in
    W: one difference is exact up to the sums' rounding)."""
    rows, out, inp = 200, 48, 64
    d, x8, off, ds, xs = wgrad_case(6, [0, rows], rows, out, inp, "bf16", "dense")
    G = torch.empty(1, out, inp, device=DEV)
    run_wgrad(d, x8, G, off)
    V = np.random.default_rng(1).normal(size=(out, inp))
    f = lambda W: float(np.sum(ds * (xs @ W.T)))
    _, size = R.weight_grads(ds, xs, [0, rows])
    tol = float((wgrad_bound(size, f64(G), [0, rows], U) * np.abs(V)).sum())
    assert abs(float((f64(G)[0] * V).sum()) - (f(0.5 * V) - f(-0.5 * V))) <= tol


@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("dy", ["bf16", "f32"])
@pytest.mark.parametrize("offsets,out,inp", [([0, 9000], 256, 512), ([0, 5000, 5001, 12000], 320, 384),
                                             ([0, 40000], 32, 128), ([0, 3000, 6100], 700, 1000)])
def test_weight_grad_many_tokens(offsets, out, inp, dy, grad):
    """Long sums: tokens cut into slices (few tiles) and chunks (fp32 sums), with
    and without what G holds already."""
    rows = offsets[-1]
    d, x8, off, ds, xs = wgrad_case(rows, offsets, rows, out, inp, dy, "dense")
    want, size = R.weight_grads(ds, xs, offsets)
    E = len(offsets) - 1
    start = torch.randn(E, out, inp, device=DEV).to(DT[grad])
    for acc in (False, True):
        G = start.clone()
        assert run_wgrad(d, x8, G, off, acc=acc) == 0
        total = want + f64(start) if acc else want
        # a chunk's sum is added to G with a rounding of its own
        extra = (np.diff(offsets) / 1024 + 2)[:, None, None] * U * (size + np.abs(total))
        within(f64(G), total, wgrad_bound(size, total, offsets, HALF[grad]) + extra)


def test_weight_grad_long_fp32_sums_stay_exact():
    """32000 tokens: the error against 64 bits stays below 3e-6 of the result
    (128 truncating additions of the tensor core lose 1.4e-6, chunks add with
    rounding)."""
    rows, out, inp = 32000, 256, 256
    d, x8, off, ds, xs = wgrad_case(7, [0, rows], rows, out, inp, "bf16", "dense")
    G = torch.empty(1, out, inp, device=DEV)
    run_wgrad(d, x8, G, off)
    want = ds.T @ xs
    assert np.linalg.norm(f64(G)[0] - want) <= 3e-6 * np.linalg.norm(want)


@pytest.mark.parametrize("dy", ["bf16", "f32"])
@pytest.mark.parametrize("E,out,inp,slices", [(64, 256, 256, False), (6, 256, 512, True)])
def test_weight_grad_long_fp32_sums_of_one_hot_expert(E, out, inp, slices, dy):
    """One expert with nearly all of 16384 tokens: the bound on the error's norm is
    that of one expert alone, whatever the average is; with and without slices."""
    rows, hot = 16384, E // 2
    offsets = [0] + np.cumsum([rows - 6 * (E - 1) if e == hot else 6 for e in range(E)]).tolist()
    d, x8, off, ds, xs = wgrad_case(13, offsets, rows, out, inp, dy, "dense")
    need = m.muon_act8_weight_grad_workspace_size(rows, out, inp, E, d.dtype, torch.float32)
    assert (need > rows * out * (6 if dy == "f32" else 2) + 256) == slices
    G = torch.empty(E, out, inp, device=DEV)
    assert run_wgrad(d, x8, G, off) == 0
    want, _ = R.weight_grads(ds, xs, offsets)
    for e in range(E):
        err = np.linalg.norm(f64(G[e]) - want[e]) / np.linalg.norm(want[e])
        assert err <= 3e-6, (e, err)


@pytest.mark.parametrize("dy", ["bf16", "f32"])
def test_weight_grad_hot_expert_of_many_chunks(dy):
    """70000 tokens, all but a few on one of 40 experts: more chunks of one tile than
    are announced at a time, between experts of one chunk and of none."""
    rows, E, out, inp, hot = 70000, 40, 40, 96, 17
    sizes = [3 if e % 3 else 0 for e in range(E)]
    sizes[hot] = rows - sum(sizes) + sizes[hot]
    offsets = [0] + np.cumsum(sizes).tolist()
    d, x8, off, ds, xs = wgrad_case(14, offsets, rows, out, inp, dy, "dense")
    want, size = R.weight_grads(ds, xs, offsets)
    start = torch.randn(E, out, inp, device=DEV)
    for acc in (False, True):
        G = start.clone()
        assert run_wgrad(d, x8, G, off, acc=acc) == 0
        total = want + f64(start) if acc else want
        for e in range(E):
            if sizes[e] == 0:
                assert torch.equal(G[e], start[e] if acc else torch.zeros_like(G[e]))
                continue
            assert np.linalg.norm(f64(G[e]) - total[e]) <= 3e-6 * (np.linalg.norm(want[e]) + np.linalg.norm(total[e])), e


def test_weight_grad_pointer_array_alignment():
    """Pointers of a device array: 16-byte steps are written, others flagged and
    their matrices left alone."""
    offsets, rows, out, inp = [0, 40, 90, 130], 130, 64, 128
    d, x8, off, ds, xs = wgrad_case(8, offsets, rows, out, inp, "bf16", "dense")
    want, size = R.weight_grads(ds, xs, offsets)
    buf = torch.full((3 * out * inp + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    n = out * inp
    for lead, flag in (((0, 8, 24), 0), ((0, 8, 17), m.MUON_FLAG_MISALIGNED)):
        buf.fill_(7.0)
        mats = [buf[e * n + lead[e]:][:n].view(out, inp) for e in range(3)]
        grp = m.Group(mats, mats, mats)
        ws = m.workspace(m.muon_act8_weight_grad_workspace_size(rows, out, inp, 3))
        m.muon_act8_weight_grad(d, x8, grp, ws, offsets=off)
        code, flags = m.muon_get_status(ws)
        assert code == m.MUON_OK and flags == flag
        for e in range(3):
            if flag and e == 2:
                assert (mats[e] == 7.0).all()
            else:
                within(f64(mats[e]), want[e], wgrad_bound(size, want, offsets, HALF["bf16"])[e])


def test_weight_grad_pointer_array_alignment_in_slices():
    """The same where the tokens of a tile are cut into slices."""
    rows, out, inp = 4096, 64, 128
    d, x8, off, ds, xs = wgrad_case(9, [0, rows], rows, out, inp, "bf16", "dense")
    want, size = R.weight_grads(ds, xs, [0, rows])
    need = m.muon_act8_weight_grad_workspace_size(rows, out, inp, 1)
    assert need > 4 * 256 * 256 * 4   # slices leave partial sums
    buf = torch.empty(out * inp + 16, dtype=torch.bfloat16, device=DEV)
    for lead, flag in ((8, 0), (1, m.MUON_FLAG_MISALIGNED)):
        buf.fill_(7.0)
        mats = [buf[lead:][: out * inp].view(out, inp)]
        ws = m.workspace(need)
        m.muon_act8_weight_grad(d, x8, m.Group(mats, mats, mats), ws, offsets=off)
        assert m.muon_get_status(ws) == (m.MUON_OK, flag)
        if flag:
            assert (buf == 7.0).all()
        else:
            within(f64(mats[0]), want[0], wgrad_bound(size, want, [0, rows], HALF["bf16"])[0])


def test_weight_grad_workspace_reused():
    """One workspace for calls that keep a copy of dy in it (fp32, rows off
    16-byte boundaries) and calls that do not, back to back on a side stream:
    each call's status is its own, each result that of a fresh workspace."""
    offsets, rows, out, inp = [0, 40, 40, 171], 171, 72, 128
    cases = []
    for k, (dy, how) in enumerate([("f32", "dense"), ("bf16", "shifted"), ("bf16", "padded"), ("f32", "shifted")]):
        d, x8, off, _, _ = wgrad_case(20 + k, offsets, rows, out, inp, dy, how)
        alone = torch.empty(3, out, inp, device=DEV)
        assert run_wgrad(d, x8, alone, off) == 0
        cases.append((d, x8, off, alone))
    ws = m.workspace(m.muon_act8_weight_grad_workspace_size(rows, out, inp, 3, torch.float32, torch.float32))
    ws.fill_(255)
    buf = torch.empty(3 * out * inp + 8, device=DEV)
    bad = [buf[e * out * inp + (e == 1):][: out * inp].view(out, inp) for e in range(3)]   # the second off its step
    group = m.Group(bad, bad, bad)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for d, x8, off, alone in cases * 3:
            G = torch.full((3, out, inp), 3.0, device=DEV)
            m.muon_act8_weight_grad(d, x8, G, ws, offsets=off)
            assert m.muon_get_status(ws) == (m.MUON_OK, 0)
            assert torch.equal(G, alone)
            m.muon_act8_weight_grad(d, x8, group, ws, offsets=off)
            assert m.muon_get_status(ws) == (m.MUON_OK, m.MUON_FLAG_MISALIGNED)
    torch.cuda.current_stream().wait_stream(side)


def test_calls_in_a_graph():
    """Every operator captured once and replayed on other inputs."""
    T, E, D, F = 300, 6, 96, 136
    g = torch.Generator(device=DEV).manual_seed(11)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)
    logits, x, gate, up, dh = rand(T, E), rand(T, D), rand(T, F), rand(T, F), rand(T, F)
    chosen = torch.topk(logits, 2).indices
    begin = torch.tensor([0, 100, T], dtype=torch.int32, device=DEV)
    offsets = torch.tensor([0, 40, 40, 130, 200, 260, T], dtype=torch.int32, device=DEV)
    loss, counts, load = rand(1), torch.empty(E, dtype=torch.int32, device=DEV), rand(2, E)
    outs = [loss, counts, load, rand(T, E), rand(T, F), rand(T, F), rand(T, F), rand(T, D), rand(E, F, D),
            rand(1, E, D)]
    x8, g8, u8 = (m.act8_empty(T, n) for n in (D, F, F))
    wb = m.workspace(m.muon_balance_workspace_size(T, E, 2))
    size = m.muon_act8_weight_grad_workspace_size
    wg = m.workspace(size(T, F, D, E, torch.float32, torch.float32))
    wr = m.workspace(size(T, E, D, 1, torch.float32, torch.float32))

    def calls():
        b = m.Balance(logits, chosen, begin)
        m.muon_balance_forward(b, loss, counts, load, wb)
        m.muon_balance_backward(b, load, outs[3])
        m.muon_act8_pack(x, x8)
        m.muon_act8_unpack(x8, outs[7])
        m.muon_act8_swiglu_forward(gate, up, outs[4], g8, u8)
        m.muon_act8_swiglu_backward(dh, g8, u8, outs[5], outs[6])
        m.muon_act8_weight_grad(outs[5], x8, outs[8], wg, offsets=offsets)
        m.muon_act8_weight_grad(outs[3], x8, outs[9], wr)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        for t in (logits, x, gate, up, dh):
            t.copy_(rand(*t.shape))
        chosen.copy_(torch.topk(logits, 2).indices)
        calls()
        want = [o.clone() for o in outs]
        for o in outs:
            o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert m.muon_get_status(wg) == (m.MUON_OK, 0)


def test_step_from_router_to_muon():
    """The operators in one step: counts -> offsets -> expert gradients into a
    group's G, which the optimizer step takes; the dense form in fp32 agrees."""
    g = torch.Generator(device=DEV).manual_seed(3)
    T, E, D, F = 192, 4, 64, 128
    x = torch.randn(T, D, generator=g, device=DEV).bfloat16()
    logits = torch.randn(T, E, generator=g, device=DEV)
    chosen = logits.argmax(dim=1, keepdim=True)
    loss, counts = torch.empty(1, device=DEV), torch.empty(E, dtype=torch.int32, device=DEV)
    load = torch.empty(1, E, device=DEV)
    ws = m.workspace(m.muon_balance_workspace_size(T, E))
    m.muon_balance_forward(m.Balance(logits, chosen), loss, counts, load, ws)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    order = torch.argsort(chosen[:, 0], stable=True)
    assert counts.sum().item() == T
    xs, dy = x[order], torch.randn(T, F, generator=g, device=DEV).bfloat16()
    x8 = m.act8_empty(T, D)
    m.muon_act8_pack(xs, x8)
    W, M = torch.randn(E, F, D, device=DEV), torch.zeros(E, F, D, device=DEV)
    G = torch.empty(E, F, D, dtype=torch.bfloat16, device=DEV)
    grp = m.Group.stacked(W, G, M)
    wg = m.workspace(m.muon_act8_weight_grad_workspace_size(T, F, D, E))
    m.muon_act8_weight_grad(dy, x8, grp, wg, offsets=offsets)
    back = torch.empty(T, D, device=DEV)
    m.muon_act8_unpack(x8, back)
    want, size = R.weight_grads(f64(dy), f64(back), offsets.tolist())
    within(f64(G), want, wgrad_bound(size, want, offsets.tolist(), HALF["bf16"]))
    before = W.clone()
    wm = m.workspace(m.muon_step_workspace_size([grp]))
    m.muon_step_batched([grp], m.hparams(), wm)
    assert m.muon_get_status(wm) == (m.MUON_OK, 0)
    assert torch.equal(M, G.float()) and not torch.equal(W, before)
