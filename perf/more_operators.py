"""Cases that measure the operators between a router's choice and the optimizer step.

Four operators of a mixture-of-experts (or dense) transformer's training step:

  sort      the copies of the tokens (one for each expert that a token was sent to)
            in the order of their experts: where each expert's rows begin, which copy
            a row holds, and which row a copy is in
  dispatch  the tokens' activations written to those rows, also as an 8-bit checkpoint,
            and the gradient of that: every token's rows added up
  combine   every token's rows multiplied by the router's weights and added up, and
            the gradients of the rows and of the weights
  norm      the norm of all gradients of a model together, and the factor that clips it

Where ``own`` is false, ``run`` computes them in elementary torch operations in
32 bits; where it is true it makes the calls a user makes.
"""
import math

import torch

own = False

BLOCK = 32           # columns that share one scale of a checkpoint
MAX_NORM = 1.0
TINY = 1e-6          # added to the norm that the clipping factor divides by
# x, the layer's input and output, and the experts' rows
_DT = {"bf16": (torch.bfloat16, torch.bfloat16), "f32": (torch.float32, torch.float32),
       "mixed": (torch.float32, torch.bfloat16)}


def _package():
    import newton_schulz_02_gb300
    return newton_schulz_02_gb300


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one short prompt through a small router: latency is all there is
        dict(name="sort-few-tokens", op="sort", tokens=33, experts=8, topk=2, index="i64", padding=False),
        # a whole batch through the router of the 256-expert layer, with padding tokens
        dict(name="sort-whole-batch", op="sort", tokens=131072, experts=256, topk=8, index="i64", padding=True),
        # a few tokens of a small layer, fp32, odd width
        dict(name="dispatch-few-tokens", op="dispatch", way="forward", tokens=61, experts=8, topk=2,
             width=1531, dtype="f32", checkpoint=False, padding=False),
        # the residual stream entering the 256-expert layer (width 7168), its checkpoint kept
        dict(name="dispatch-checkpoint", op="dispatch", way="forward", tokens=4096, experts=256, topk=8,
             width=7168, dtype="mixed", checkpoint=True, padding=False),
        # the same layer, a whole batch, no checkpoint
        dict(name="dispatch-batch", op="dispatch", way="forward", tokens=16384, experts=256, topk=8,
             width=7168, dtype="bf16", checkpoint=False, padding=False),
        # its gradient, padding tokens among the others
        dict(name="dispatch-gradient", op="dispatch", way="gradient", tokens=16384, experts=256, topk=8,
             width=7168, dtype="bf16", checkpoint=False, padding=True),
        # a few tokens of a layer with many experts: one step of generation
        dict(name="combine-few-tokens", op="combine", way="forward", tokens=7, experts=256, topk=8,
             width=2048, weights="f32", dtype="bf16", padding=False),
        # the output of the 256-expert layer, a whole batch, added up in fp32
        dict(name="combine-batch", op="combine", way="forward", tokens=16384, experts=256, topk=8,
             width=7168, weights="f32", dtype="mixed", padding=False),
        # a small fp32 layer of odd width whose padding tokens go nowhere
        dict(name="combine-gradient-odd", op="combine", way="gradient", tokens=1023, experts=60, topk=6,
             width=1111, weights="f32", dtype="f32", padding=True),
        # the gradients of the 256-expert layer's output, a whole batch
        dict(name="combine-gradient-batch", op="combine", way="gradient", tokens=16384, experts=256,
             topk=8, width=7168, weights="f32", dtype="bf16", padding=False),
        # one small layer in fp32, its norm below the limit: nothing is clipped
        dict(name="norm-small", op="norm", layers=1, width=256, inner=512, kv=128, vocab=0, experts=0,
             dtype="f32", size=1e-4),
        # eight layers of the dense model (14336 x 4096 and its attention), bf16
        dict(name="norm-dense", op="norm", layers=8, width=4096, inner=14336, kv=1024, vocab=0, experts=0,
             dtype="bf16", size=1e-3),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _parameters(case):
    """Values in all of a norm case's tensors."""
    return sum(math.prod(s) for s, _ in _shapes(case))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "dispatch", "combine", "combine", "norm"])
    if op == "norm":
        experts = rng.choice([0, 0, 4, 16])
        while True:
            c = dict(op=op, layers=rng.randint(1, 8), width=8 * _between(rng, 8, 512),
                     inner=8 * _between(rng, 8, 1792), kv=8 * _between(rng, 1, 128),
                     vocab=rng.choice([0, _between(rng, 100, 50000)]), experts=experts,
                     dtype=rng.choice(["bf16", "f32"]), size=10.0 ** rng.uniform(-7, 1))
            if _parameters(c) * (1 if c["dtype"] == "bf16" else 2) <= 17 * 10 ** 8:
                return c
    experts = rng.choice([4, 8, 16, 17, 60, 64, 128, 160, 256, 384, 512])
    topk = rng.randint(1, min(8, experts))
    if op == "sort":
        return dict(op=op, tokens=_between(rng, 1, 131072), experts=experts, topk=topk,
                    index=rng.choice(["i32", "i64"]), padding=rng.random() < 0.5)
    width = _between(rng, 1, 16384)
    if rng.random() < 0.6 and width >= 64:
        width -= width % 64
    dtype = rng.choice(["bf16", "bf16", "f32", "mixed"])
    way = rng.choice(["forward", "gradient"])
    most = 16384 * 8 * 7168 // (1 if dtype == "bf16" else 2)
    case = dict(op=op, way=way, experts=experts, topk=topk, width=width, dtype=dtype)
    if op == "dispatch":
        case["checkpoint"] = way == "forward" and rng.random() < 0.4
        case["padding"] = not case["checkpoint"] and rng.random() < 0.5
        most //= 4 if case["checkpoint"] else 1
    else:
        case["weights"] = rng.choice(["f32", "f32", "bf16"])
        case["padding"] = rng.random() < 0.5
    case["tokens"] = _between(rng, 1, max(1, min(131072, most // (topk * width))))
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=g.device, dtype=torch.float32)


def _activation(g, rows, cols, dtype):
    """Unit-scale values whose tokens differ in size and with a few outlier channels."""
    x = _normal(g, rows, cols)
    x *= torch.exp(0.3 * _normal(g, rows, 1))
    x *= torch.where(torch.rand(1, cols, generator=g, device=g.device) < 0.005, 15.0, 1.0)
    return x.to(dtype)


def _router(case, g):
    """Choices [tokens, topk] of a router whose experts are not equally liked, its weights,
    and which tokens are valid (None: all)."""
    T, E, K = case["tokens"], case["experts"], case["topk"]
    logits = 1.5 * _normal(g, T, E) + _normal(g, 1, E)
    top = torch.topk(logits, K, dim=1)
    weights = top.values.softmax(dim=1)
    mask = torch.rand(T, generator=g, device=g.device) > 0.1 if case["padding"] else None
    return top.indices, weights, mask


def _plan(chosen, mask, experts):
    """offsets [experts + 1], order and place of the tokens' copies."""
    T, K = chosen.shape
    key = chosen.flatten().long()
    if mask is not None:
        key = torch.where(mask.repeat_interleave(K), key, torch.full_like(key, experts))
    order = torch.sort(key, stable=True).indices
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=key.device)
    offsets[1:] = torch.cumsum(torch.bincount(key, minlength=experts + 1)[:experts], 0)
    row = torch.arange(T * K, dtype=torch.int32, device=key.device)
    inside = row < offsets[-1]
    place = torch.empty_like(row)
    place[order] = torch.where(inside, row, torch.full_like(row, -1))
    order = torch.where(inside, order.to(torch.int32), torch.full_like(row, -1))
    return offsets, order, place.view(T, K)


def _shapes(case):
    """Shapes (stacked matrices, or stacked vectors) and types of a model's gradients."""
    n, d, f, dt = case["layers"], case["width"], case["inner"], case["dtype"]
    mlp = n * max(1, case["experts"])
    out = [((n, d, d), dt), ((n, case["kv"], d), dt), ((n, case["kv"], d), dt), ((n, d, d), dt),
           ((mlp, f, d), dt), ((mlp, f, d), dt), ((mlp, d, f), dt), ((2 * n, d), "f32")]
    if case["vocab"]:
        out.append(((case["vocab"], d), dt))
    if case["experts"]:
        out.append(((n, case["experts"], d), "f32"))
    return out


def _gradients(case, seed):
    """A model's gradients: normal values, each tensor of a size of its own."""
    g = torch.Generator(device=_device()).manual_seed(seed)
    size = case["size"] * torch.exp(0.5 * torch.randn(16, generator=torch.Generator().manual_seed(seed)))
    return [torch.empty(shape, dtype=_DT[dt][0], device=g.device).normal_(0.0, float(size[i]), generator=g)
            for i, (shape, dt) in enumerate(_shapes(case))]


def prepare(case, seed):
    dev, op = _device(), case["op"]
    s = dict(case=case)
    if op == "norm":
        s["grads"] = _gradients(case, seed)
        s["norm"], s["scale"] = torch.empty(1, device=dev), torch.empty(1, device=dev)
        if own:   # a training program lists its gradients once
            m = _package()
            s["list"] = m.Grads(s["grads"])
            s["ws"] = m.workspace(m.muon_grad_norm_workspace_size(s["list"]), dev)
        return s
    g = torch.Generator(device=dev).manual_seed(seed)
    T, E, K = case["tokens"], case["experts"], case["topk"]
    chosen, weights, mask = _router(case, g)
    if op == "sort":
        s["chosen"] = chosen.to(torch.int64 if case["index"] == "i64" else torch.int32)
        s["mask"] = mask
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=dev)
        s["order"] = torch.full((T * K,), -1, dtype=torch.int32, device=dev)
        s["place"] = torch.empty(T, K, dtype=torch.int32, device=dev)
        if own:
            m = _package()
            s["routing"] = m.Routing(s["offsets"], s["order"], s["place"])
            s["ws"] = m.workspace(m.muon_moe_sort_workspace_size(T, E, K), dev)
        return s
    # the plan that the sort left, and the activations of both sides of the layer
    s["offsets"], s["order"], s["place"] = _plan(chosen, mask, E)
    s["rows"] = int(s["offsets"][-1])
    if own:
        s["routing"] = _package().Routing(s["offsets"], s["order"], s["place"])
    D, (outer, inner) = case["width"], _DT[case["dtype"]]
    if op == "dispatch" and case["way"] == "forward":
        s["x"] = _activation(g, T, D, outer)
        s["xs"] = torch.zeros(T * K, D, dtype=inner, device=dev)
        if case["checkpoint"]:
            s["values"] = torch.zeros(T * K, D, dtype=torch.bfloat16, device=dev)
    elif op == "dispatch":
        s["dxs"] = (1e-3 * _activation(g, T * K, D, torch.float32)).to(inner)
        s["dx"] = torch.empty(T, D, dtype=outer, device=dev)
    else:
        s["weights"] = weights.to(_DT[case["weights"]][0])
        s["ys"] = _activation(g, T * K, D, inner)
        if case["way"] == "forward":
            s["out"] = torch.empty(T, D, dtype=outer, device=dev)
        else:
            s["dout"] = (1e-3 * _activation(g, T, D, torch.float32)).to(outer)
            s["dys"] = torch.zeros(T * K, D, dtype=inner, device=dev)
            s["dweights"] = torch.empty_like(s["weights"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _quantised(x):
    """The values that a checkpoint of x holds: the scale of 32 columns is the
    smallest power of two whose 127-fold reaches their largest magnitude."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    xp = torch.zeros(rows, nb * BLOCK, dtype=torch.float32, device=x.device)
    xp[:, :cols] = x
    xb = xp.view(rows, nb, BLOCK)
    m, k = torch.frexp(xb.abs().amax(dim=2))        # amax = m * 2^k, 1/2 <= m < 1
    e = torch.where(m > 127 / 128, k - 6, k - 7)
    e = torch.where(m == 0, torch.full_like(e, -126), e).clamp(min=-126)[:, :, None]
    return torch.ldexp(torch.round(torch.ldexp(xb, -e)), e).flatten(1)[:, :cols]


def _rows_of(y, place):
    """y's rows at `place` [tokens, topk] in 32 bits, 0 where a copy has no row."""
    taken = y.float()[place.clamp(min=0).long()]
    return torch.where((place >= 0)[:, :, None], taken, torch.zeros((), device=y.device))


def _plain_dispatch(s):
    n, source = s["rows"], s["order"][: s["rows"]].long() // s["case"]["topk"]
    if s["case"]["way"] == "gradient":
        return dict(dx=_rows_of(s["dxs"], s["place"]).sum(dim=1).to(s["dx"].dtype))
    x = s["x"].float()
    xs = torch.zeros_like(s["xs"])
    xs[:n] = x[source].to(xs.dtype)
    if not s["case"]["checkpoint"]:
        return dict(xs=xs)
    values = torch.zeros_like(s["values"])
    values[:n] = _quantised(x)[source].to(values.dtype)
    return dict(xs=xs, values=values)


def _plain_combine(s):
    w = s["weights"].float()
    if s["case"]["way"] == "forward":
        return dict(out=(w[:, :, None] * _rows_of(s["ys"], s["place"])).sum(dim=1).to(s["out"].dtype))
    n, copy = s["rows"], s["order"][: s["rows"]].long()
    source = copy // s["case"]["topk"]
    dout = s["dout"].float()[source]
    dys = torch.zeros_like(s["dys"])
    dys[:n] = (w.flatten()[copy][:, None] * dout).to(dys.dtype)
    dw = torch.zeros(w.numel(), device=w.device)
    dw[copy] = (dout * s["ys"][:n].float()).sum(dim=1)
    return dict(dys=dys, dweights=dw.view_as(w).to(s["weights"].dtype))


def _plain_norm(s):
    squares = [t.float().square().sum(dtype=torch.float64) for t in s["grads"]]
    norm = torch.stack(squares).sum().sqrt().reshape(1)
    return dict(norm=norm.float(), scale=(MAX_NORM / (norm + TINY)).clamp(max=1.0).float())


def run(s):
    op, case = s["case"]["op"], s["case"]
    if not own:
        if op == "sort":
            return dict(zip(("offsets", "order", "place"), _plan(s["chosen"], s["mask"], case["experts"])))
        return {"dispatch": _plain_dispatch, "combine": _plain_combine, "norm": _plain_norm}[op](s)
    m = _package()
    if op == "norm":
        m.muon_grad_norm(s["list"], s["norm"], s["scale"], s["ws"], max_norm=MAX_NORM)
        return dict(norm=s["norm"], scale=s["scale"])
    r = s["routing"]
    if op == "sort":
        m.muon_moe_sort(s["chosen"], r, s["ws"], mask=s["mask"])
        return dict(offsets=s["offsets"], order=s["order"], place=s["place"])
    if op == "dispatch":
        if case["way"] == "gradient":
            m.muon_moe_dispatch_backward(s["dxs"], r, s["dx"])
            return dict(dx=s["dx"])
        if not case["checkpoint"]:
            m.muon_moe_dispatch(s["x"], r, s["xs"])
            return dict(xs=s["xs"])
        x8 = m.act8_empty(*s["xs"].shape, device=s["x"].device)
        m.muon_moe_dispatch(s["x"], r, s["xs"], x8)
        m.muon_act8_unpack(x8, s["values"])
        return dict(xs=s["xs"], values=s["values"])
    if case["way"] == "forward":
        m.muon_moe_combine(s["ys"], s["weights"], r, s["out"])
        return dict(out=s["out"])
    m.muon_moe_combine_backward(s["dout"], s["ys"], s["weights"], r, s["dys"], s["dweights"])
    return dict(dys=s["dys"], dweights=s["dweights"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "norm":
        values = [(math.prod(s), 2 if dt == "bf16" else 4) for s, dt in _shapes(case)]
        return dict(bytes=sum(n * b for n, b in values), flops=2 * sum(n for n, _ in values))
    copies = case["tokens"] * case["topk"]
    held = copies * (0.9 if case["padding"] else 1.0)      # copies that have a row
    if case["op"] == "sort":
        # the choices are read; the row of every copy and the copy of every row are written
        return dict(bytes=held * (4 if case["index"] == "i32" else 8) + 4 * (copies + held)
                    + 4 * case["experts"], flops=copies)
    outer, inner = (2 if t == torch.bfloat16 else 4 for t in _DT[case["dtype"]])
    tokens, rows = case["tokens"] * case["width"], held * case["width"]
    if case["op"] == "dispatch":
        kept = rows * (1 + 1 / BLOCK) if case["checkpoint"] else 0.0
        # a checkpoint is written, and its values are read back in 16 bits
        return dict(bytes=tokens * outer + rows * inner + 4 * copies + 2 * kept
                    + (2 * rows if kept else 0), flops=rows)
    if case["way"] == "forward":
        return dict(bytes=rows * inner + tokens * outer + 8 * copies, flops=2 * rows)
    return dict(bytes=2 * rows * inner + tokens * outer + 12 * copies, flops=3 * rows)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_quantised(x):
    """Each value to the nearest multiple (ties to even) of 2^e, e the least integer
    >= -126 with 127 * 2^e >= the largest magnitude among its 32 columns."""
    rows, cols = x.shape
    y = torch.nn.functional.pad(x, (0, -cols % BLOCK)).reshape(rows, -1, BLOCK)
    big = y.abs().max(dim=2, keepdim=True).values
    e = torch.ceil(torch.log2(torch.clamp(big, min=2.0 ** -126) / 127))
    e = torch.where(127 * torch.exp2(e) < big, e + 1, e)        # the logarithm's own rounding
    e = torch.where(127 * torch.exp2(e - 1) >= big, e - 1, e).clamp(min=-126)
    step = torch.exp2(e)
    return (torch.round(y / step) * step).reshape(rows, -1)[:, :cols]


def _exact_sort(case, seed):
    """Expert by expert: the copies of an expert in their own order."""
    s = prepare(case, seed)
    T, K, E = case["tokens"], case["topk"], case["experts"]
    flat = s["chosen"].cpu().long().flatten()
    if s["mask"] is not None:
        flat[~s["mask"].cpu().repeat_interleave(K)] = -1
    order = torch.full((T * K,), -1, dtype=torch.int32)
    place = torch.full((T * K,), -1, dtype=torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    at = 0
    for e in range(E):
        here = torch.nonzero(flat == e).flatten()
        order[at: at + len(here)] = here.to(torch.int32)
        place[here] = torch.arange(at, at + len(here), dtype=torch.int32)
        at += len(here)
        offsets[e + 1] = at
    return dict(offsets=offsets, order=order, place=place.view(T, K))


def _exact_layer(case, seed):
    """Choice by choice: what the copies of the tokens' k-th choices give and get."""
    s = prepare(case, seed)
    T, K, D = case["tokens"], case["topk"], case["width"]
    forward = case["way"] == "forward"
    f64 = dict(dtype=torch.float64, device=s["place"].device)
    held = [torch.nonzero(s["place"][:, k] >= 0).flatten() for k in range(K)]
    if case["op"] == "dispatch" and forward:
        x = s["x"].double()
        out = dict(xs=torch.zeros(T * K, D, **f64))
        if case["checkpoint"]:
            out["values"], q = torch.zeros(T * K, D, **f64), _exact_quantised(x)
        for k, t in enumerate(held):
            out["xs"][s["place"][t, k].long()] = x[t]
            if case["checkpoint"]:
                out["values"][s["place"][t, k].long()] = q[t]
        return out
    if case["op"] == "dispatch":
        dx = torch.zeros(T, D, **f64)
        for k, t in enumerate(held):
            dx[t] += s["dxs"][s["place"][t, k].long()].double()
        return dict(dx=dx)
    w = s["weights"].double()
    if forward:
        out = torch.zeros(T, D, **f64)
        for k, t in enumerate(held):
            out[t] += w[t, k, None] * s["ys"][s["place"][t, k].long()].double()
        return dict(out=out)
    dout = s["dout"].double()
    dys, dw = torch.zeros(T * K, D, **f64), torch.zeros(T, K, **f64)
    for k, t in enumerate(held):
        rows = s["place"][t, k].long()
        dys[rows] = w[t, k, None] * dout[t]
        dw[t, k] = torch.einsum("td,td->t", dout[t], s["ys"][rows].double())
    return dict(dys=dys, dweights=dw)


def exact(case, seed):
    if case["op"] == "sort":
        return _exact_sort(case, seed)
    if case["op"] != "norm":
        return _exact_layer(case, seed)
    total = torch.zeros((), dtype=torch.float64, device=_device())
    for t in _gradients(case, seed):
        for part in t.flatten().split(1 << 26):
            total += torch.dot(part.double(), part.double())
    norm = total.sqrt().reshape(1)
    return dict(norm=norm, scale=torch.minimum(torch.ones_like(norm), MAX_NORM / (norm + TINY)))
