"""The norm of all gradients and the steps that take its clipping factor, on the
GPU against the float64 oracle.

Tolerance of the norm: 32 squares are added in fp32 (at most 10 roundings in a
chain and one for the square: 11 U relative, all terms positive; 64 of bf16, whose
squares are exact, with 11), the rest in 48 bits; a root halves that, and the result
is rounded: 7 U.  The factor: the same and two roundings."""
import math

import numpy as np
import pytest
import torch

import newton_schulz_02_gb300 as m
from oracle import moe_ref as R
from tests.gpu_util import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    m.load_library()
    torch.cuda.set_device(0)


def run(items, max_norm=math.inf, ws=None):
    g = m.Grads(items)
    norm, scale = torch.full((1,), 5.0, device=DEV), torch.full((1,), 5.0, device=DEV)
    if ws is None:
        ws = m.workspace(m.muon_grad_norm_workspace_size(g))
        ws.fill_(255)
    m.muon_grad_norm(g, norm, scale, ws, max_norm=max_norm)
    code, flags = m.muon_get_status(ws)
    assert code == m.MUON_OK
    return norm, scale, flags


def check(items, tensors, max_norm=math.inf):
    norm, scale, flags = run(items, max_norm)
    n, s = R.grad_norm([f64(t) for t in tensors], max_norm)
    assert flags == 0
    assert abs(norm.item() - n) <= 7 * U * n + 2.0 ** -150
    assert abs(scale.item() - s) <= 9 * U * s
    return norm, scale


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("numel", [1, 7, 8, 9, 255, 8191, 8192, 8193, 70001, 3000003])
def test_norm_of_one_tensor(dtype, numel):
    t = torch.randn(numel, device=DEV).to(dtype)
    check([t], [t], max_norm=0.5)


def test_norm_of_groups_tensors_and_views():
    """Matrices of a Muon group (heads of a wider weight among them), AdamW tensors of odd
    sizes, more groups than one launch takes, and tensors in no group."""
    rand = lambda *s, dt=torch.float32: torch.randn(*s, device=DEV).to(dt)
    W, G, M = rand(3, 64, 200, dt=torch.bfloat16), rand(3, 64, 200, dt=torch.bfloat16), rand(3, 64, 200)
    items, tensors = [m.Group.stacked(W, G, M)], [G]
    Wh, Gh, Mh = rand(96, 4 * 48), rand(96, 4 * 48), rand(96, 4 * 48)
    heads = m.Group.split_head(Wh, Gh, Mh, 4, 48)
    items.append(heads)
    tensors.append(Gh)
    part = m.Group([Wh[:, 48:96]], [Gh[:, 48:96]], [Mh[:, 48:96]])     # one head once more
    items.append(part)
    tensors.append(Gh[:, 48:96])
    a = [rand(n) for n in (5, 1001, 5, 4096)]
    items += m.adamw_groups(a, a, a, a)
    tensors += a
    check(items, tensors, max_norm=3.0)
    free = [rand(k + 1, dt=torch.bfloat16 if k % 2 else torch.float32) for k in range(150)]
    check(items + free, tensors + free, max_norm=3.0)
    check([torch.empty(0, device=DEV), free[3]], [free[3]])


def test_strided_matrices_larger_than_a_piece():
    big = torch.randn(700, 1000, device=DEV)
    for view in (big[:, 8:992], big[3:, :8], big[:, :504]):
        z = torch.zeros_like(view)
        g = m.Group([view], [view], [view])
        check([g], [view], max_norm=1.0)


@pytest.mark.parametrize("size", [1e-44, 1e-30, 1e-18, 1e-12, 1e12, 1e18, 1e30, 3e38])
def test_squares_neither_overflow_nor_vanish(size):
    t = torch.full((10007,), size, device=DEV)
    t[::3] = -size
    norm, scale, flags = run([t], max_norm=1.0)
    n, s = R.grad_norm([f64(t)], 1.0)
    if n > 3.4028235e38:     # the norm itself is out of fp32's range, its factor is not
        assert math.isinf(norm.item())
    else:
        assert abs(norm.item() - n) <= 7 * U * n + 2.0 ** -149
    assert flags == 0 and abs(scale.item() - s) <= 9 * U * s + 2.0 ** -149
    mixed = torch.randn(10007, device=DEV)
    mixed[5], mixed[9000] = size, 1e-40
    check([mixed], [mixed]) if size < 1e30 else None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [1e-3, 0.0217])
def test_norm_of_many_values_keeps_its_bound(dtype, size):
    """Half a million partial sums, whose roundings might all go one way."""
    g = torch.Generator(device=DEV).manual_seed(3)
    t = torch.empty(1 << 25, dtype=dtype, device=DEV).normal_(0.0, size, generator=g)
    n = math.sqrt(sum(torch.dot(p, p).item() for p in (q.double() for q in t.split(1 << 22))))
    norm, scale, flags = run([t], max_norm=1.0)
    assert flags == 0 and abs(norm.item() - n) <= 7 * U * n
    assert abs(scale.item() - min(1.0, 1.0 / (n + 1e-6))) <= 9 * U * min(1.0, 1.0 / (n + 1e-6))


def test_a_norm_beyond_the_range_of_fp32_still_clips():
    """The norm reads as infinity; the factor is finite, and the steps take it."""
    G = torch.full((4, 1024), 3e38, device=DEV)
    G[1, ::2] = -2.5e38
    W, mom, var = torch.rand_like(G), torch.rand_like(G), torch.rand_like(G)
    norm, scale, flags = run([G], max_norm=1.0)
    n, s = R.grad_norm([f64(G)], 1.0)
    assert n > 3.5e38 and norm.item() == math.inf and flags == 0
    assert abs(scale.item() - s) <= 9 * U * s + 2.0 ** -150
    W2, m2, v2 = W.clone(), mom.clone(), var.clone()
    m.muon_adamw_step(m.adamw_groups([W], [G], [mom], [var]), m.adamw_hparams(), grad_scale=scale)
    m.muon_adamw_step(m.adamw_groups([W2], [G * scale], [m2], [v2]), m.adamw_hparams())
    assert torch.equal(W, W2) and torch.equal(mom, m2) and torch.equal(var, v2)
    M, start = torch.zeros_like(G), W.clone()
    group = m.Group([W], [G], [M])
    ws = m.workspace(m.muon_step_workspace_size([group]))
    m.muon_step_batched([group], m.hparams(), ws, grad_scale=scale)
    assert m.muon_get_status(ws) == (m.MUON_OK, 0)
    assert torch.equal(M, G * scale) and not torch.equal(W, start)


def test_norm_of_tensors_of_more_than_32_bits_of_values():
    """Values and rows behind 2^32, dense and as columns of a wider matrix."""
    rows, width = (1 << 19) + 3, 8208
    big = torch.zeros(rows, width, dtype=torch.bfloat16, device=DEV)
    assert big.numel() > 1 << 32
    big[0, 0], big[rows - 1, width - 1], big[rows - 1, 8], big[rows // 2, 8199] = 3.0, 5.0, 2.0, 4.0
    big[rows - 1, 8200], big[7, 7] = 16.0, 1.0
    norm, _, flags = run([big])
    assert flags == 0 and abs(norm.item() - math.sqrt(9 + 25 + 4 + 16 + 256 + 1)) <= 7 * U * 18
    g = m.Grads([big])
    g.c[0] = m.muon_grads_t(1, rows, 8192, width, m.MUON_BF16, g.c[0].ptrs)
    norm, scale = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    ws = m.workspace(m.muon_grad_norm_workspace_size(g))
    m.muon_grad_norm(g, norm, scale, ws)
    assert abs(norm.item() - math.sqrt(9 + 4 + 1)) <= 7 * U * 4
    g.ptrs += 16
    m.muon_grad_norm(g, norm, scale, ws)
    assert abs(norm.item() - math.sqrt(4 + 16)) <= 7 * U * 5


def test_two_graphs_share_a_workspace():
    """Two captured norms over one workspace, replayed in turn on other gradients."""
    sets = [[torch.randn(n, device=DEV) for n in sizes] for sizes in ((9, 70001), (1 << 20, 3, 5000001))]
    grads = [m.Grads(ts) for ts in sets]
    ws = m.workspace(max(m.muon_grad_norm_workspace_size(g) for g in grads))
    out = [(torch.empty(1, device=DEV), torch.empty(1, device=DEV)) for _ in sets]
    graphs = []
    for g, (norm, scale) in zip(grads, out):
        m.muon_grad_norm(g, norm, scale, ws, max_norm=1.0)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            m.muon_grad_norm(g, norm, scale, ws, max_norm=1.0)
    for turn in range(4):
        ts, (norm, scale) = sets[turn % 2], out[turn % 2]
        ts[0].normal_()
        ts[1][0] = 1e30 if turn == 2 else 0.5
        graphs[turn % 2].replay()
        n, s = R.grad_norm([f64(t) for t in ts], 1.0)
        assert abs(norm.item() - n) <= 7 * U * n and abs(scale.item() - s) <= 9 * U * s + 2.0 ** -149


def test_zero_gradients_and_the_border_of_clipping():
    z = torch.zeros(5000, device=DEV)
    norm, scale, flags = run([z], max_norm=0.0)
    assert (norm.item(), scale.item(), flags) == (0.0, 0.0, 0)
    norm, scale, _ = run([z], max_norm=1.0)
    assert (norm.item(), scale.item()) == (0.0, 1.0)
    t = torch.full((16,), 0.25, device=DEV)     # norm 1
    assert run([t], max_norm=2.0)[1].item() == 1.0
    assert run([t], max_norm=math.inf)[1].item() == 1.0
    assert run([t], max_norm=1.0)[1].item() == np.float32(1.0 / (1.0 + 1e-6))
    assert run([t], max_norm=0.0)[1].item() == 0.0


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("at", [0, 4999, 5000])
def test_not_finite(bad, at):
    t = torch.randn(5001, device=DEV)
    t[at] = bad
    norm, scale, flags = run([torch.randn(64, device=DEV), t], max_norm=1.0)
    assert flags == m.MUON_FLAG_NONFINITE and math.isnan(scale.item())
    assert math.isnan(norm.item()) if math.isnan(bad) else norm.item() == math.inf


def test_misaligned_pointer_in_a_group_is_flagged_and_left_out():
    buf, ok = torch.randn(1000, device=DEV), torch.randn(64, 8, device=DEV)
    off = buf[1:513].view(64, 8)
    g = m.Group([ok, off], [ok, off], [ok, off])
    norm, _, flags = run([g])
    n, _ = R.grad_norm([f64(ok)])
    assert flags == m.MUON_FLAG_MISALIGNED and abs(norm.item() - n) <= 7 * U * n


def test_repeats_its_bits_streams_and_graph():
    ts = [torch.randn(n, device=DEV) for n in (100003, 7, 1 << 20)]
    g = m.Grads(ts)
    ws = m.workspace(m.muon_grad_norm_workspace_size(g))
    norm, scale = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    m.muon_grad_norm(g, norm, scale, ws, max_norm=1.0)
    first = (norm.item(), scale.item())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.muon_grad_norm(g, norm, scale, ws, max_norm=1.0, stream=side)
    torch.cuda.synchronize()
    assert (norm.item(), scale.item()) == first
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.muon_grad_norm(g, norm, scale, ws, max_norm=1.0)
    for _ in range(2):
        norm.zero_()
        graph.replay()
        assert (norm.item(), scale.item()) == first
    ts[0].mul_(2.0)
    graph.replay()
    n, _ = R.grad_norm([f64(t) for t in ts])
    assert abs(norm.item() - n) <= 7 * U * n


# ---- the steps --------------------------------------------------------------
def muon_case(dtype, shape, seed=0, heads=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda: torch.randn(*shape, generator=g, device=DEV)
    return rand().mul_(0.02).to(dtype), rand().mul_(3.0).to(dtype), rand().abs_().mul_(1e-3)


@pytest.mark.parametrize("style", ["sgd", "ema"])
@pytest.mark.parametrize("shape", [(2, 256, 512), (2, 512, 256), (1, 64, 72), (3, 128, 1024)])
def test_muon_step_with_a_factor_is_the_step_of_the_scaled_gradient(style, shape):
    """fp32: G * scale rounded to fp32 is what torch multiplies to; the same bits follow."""
    W, G, M = muon_case(torch.float32, shape)
    scale = torch.tensor([0.0377], device=DEV)
    hp = m.hparams(style=style, lr=1e-2, t=3)
    W2, M2, G2 = W.clone(), M.clone(), G * scale
    a, b = m.Group.stacked(W, G, M), m.Group.stacked(W2, G2, M2)
    ws = m.workspace(m.muon_step_workspace_size([a]))
    keep = G.clone()
    m.muon_step_batched([a], hp, ws, grad_scale=scale)
    assert m.muon_get_status(ws) == (m.MUON_OK, 0)
    m.muon_step_batched([b], hp, ws)
    assert torch.equal(W, W2) and torch.equal(M, M2) and torch.equal(G, keep)


@pytest.mark.parametrize("shape", [(2, 256, 384), (2, 384, 256), (2, 128, 512)])
def test_muon_step_scales_bf16_gradients_in_fp32(shape):
    """bf16 G: the product is not rounded to bf16, as in a step whose G is fp32."""
    W, G, M = muon_case(torch.bfloat16, shape)
    scale = torch.tensor([0.0377], device=DEV)
    W2, M2, G2 = W.clone(), M.clone(), G.float() * scale
    a, b = m.Group.stacked(W, G, M), m.Group.stacked(W2, G2, M2)
    ws = m.workspace(m.muon_step_workspace_size([a]))
    m.muon_step_batched([a], m.hparams(), ws, grad_scale=scale)
    m.muon_step_batched([b], m.hparams(), ws)
    assert torch.equal(W, W2) and torch.equal(M, M2)


def test_steps_with_factor_one_are_the_steps_without():
    one = torch.ones(1, device=DEV)
    W, G, M = muon_case(torch.bfloat16, (2, 256, 384))
    W2, M2 = W.clone(), M.clone()
    a, b = m.Group.stacked(W, G, M), m.Group.stacked(W2, G, M2)
    ws = m.workspace(m.muon_step_workspace_size([a]))
    m.muon_step_batched([a], m.hparams(), ws, grad_scale=one)
    m.muon_step_batched([b], m.hparams(), ws)
    assert torch.equal(W, W2) and torch.equal(M, M2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_adamw_step_with_a_factor(dtype):
    """bf16 G: G * scale in fp32 is not rounded to bf16 before it is used."""
    n, scale = 10005, torch.tensor([0.0211], device=DEV)
    W, G = (torch.randn(n, device=DEV).to(dtype) for _ in range(2))
    mv = [torch.rand(n, device=DEV) for _ in range(2)]
    W2, mv2 = W.clone(), [t.clone() for t in mv]
    hp = m.adamw_hparams(lr=1e-2, t=2)
    m.muon_adamw_step(m.adamw_groups([W], [G], mv[:1], mv[1:]), hp, grad_scale=scale)
    m.muon_adamw_step(m.adamw_groups([W2], [G.float() * scale], mv2[:1], mv2[1:]), hp)
    assert torch.equal(W, W2) and torch.equal(mv[0], mv2[0]) and torch.equal(mv[1], mv2[1])


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_factor_that_is_not_finite_changes_nothing(bad):
    scale = torch.tensor([bad], device=DEV)
    for shape in ((2, 256, 512), (2, 512, 256), (2, 128, 256)):
        W, G, M = muon_case(torch.float32, shape)
        keep = [t.clone() for t in (W, G, M)]
        g = m.Group.stacked(W, G, M)
        ws = m.workspace(m.muon_step_workspace_size([g]))
        m.muon_step_batched([g], m.hparams(), ws, grad_scale=scale)
        assert m.muon_get_status(ws) == (m.MUON_OK, m.MUON_FLAG_NONFINITE)
        assert all(torch.equal(a, b) for a, b in zip(keep, (W, G, M)))
    a = [torch.rand(1003, device=DEV) for _ in range(4)]
    keep = [t.clone() for t in a]
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    m.muon_adamw_step(m.adamw_groups(*[[t] for t in a]), m.adamw_hparams(), flags, grad_scale=scale)
    assert flags.item() == m.MUON_FLAG_NONFINITE
    assert all(torch.equal(p, q) for p, q in zip(keep, a))


def test_norm_then_both_steps_in_a_graph():
    """Norm, Muon and AdamW captured together: the factor goes from one to the other on
    the device, and a replay with a NaN among the gradients changes no weight."""
    W, G, M = muon_case(torch.float32, (2, 256, 512))
    a = [torch.rand(300, device=DEV) for _ in range(4)]
    mu, ad = [m.Group.stacked(W, G, M)], m.adamw_groups(*[[t] for t in a])
    grads = m.Grads(mu + ad)
    norm, scale = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    wsn, ws = m.workspace(m.muon_grad_norm_workspace_size(grads)), m.workspace(m.muon_step_workspace_size(mu))

    def step():
        m.muon_grad_norm(grads, norm, scale, wsn, max_norm=1.0)
        m.muon_step_batched(mu, m.hparams(), ws, grad_scale=scale)
        m.muon_adamw_step(ad, m.adamw_hparams(), grad_scale=scale)

    start = [t.clone() for t in (W, M, *a)]
    step()
    torch.cuda.synchronize()
    after = [t.clone() for t in (W, M, *a)]
    n, s = R.grad_norm([f64(G), f64(a[1])], 1.0)
    assert n > 100 and abs(scale.item() - s) <= 9 * U * s
    for t, v in zip((W, M, *a), start):
        t.copy_(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, v in zip((W, M, *a), start):
        t.copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(after, (W, M, *a)))
    G[1, 7, 9] = math.nan
    graph.replay()
    torch.cuda.synchronize()
    assert math.isnan(scale.item()) and all(torch.equal(p, q) for p, q in zip(after, (W, M, *a)))
