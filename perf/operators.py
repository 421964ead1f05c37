"""Cases that measure the training-side operators next to the optimizer step.

Four operators of a mixture-of-experts (or dense) transformer's training step,
which together produce the gradients a Muon / AdamW step consumes:

  balance     the router's balance loss over packed sequences, the per-expert
              token counts, and the gradient of the logits
  checkpoint  an activation written as 8-bit codes with a power-of-two scale for
              every 32 columns of a row, and read back
  swiglu      h = silu(gate) * up with gate and up kept as 8-bit checkpoints, and
              its backward pass from them (which also rebuilds h as a checkpoint)
  wgrad       the weight gradients dW_e = dY_e^T X_e of all experts from an 8-bit
              checkpoint of X

Where ``own`` is false, ``run`` computes them in elementary torch operations in
32 bits; where it is true it makes the calls a user makes.
"""
import math

import torch

own = False

BLOCK = 32           # columns that share one scale of a checkpoint
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _package():
    import newton_schulz_02_gb300
    return newton_schulz_02_gb300


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one short prompt through a small router: latency is all there is
        dict(name="balance-few-tokens", op="balance", tokens=33, experts=8, topk=2, sequences=1,
             score="softmax", dtype="f32", index="i64", padding=False),
        # packed sequences of very different lengths (one of them empty), padding tokens,
        # two disabled experts, sigmoid scores
        dict(name="balance-packed-odd", op="balance", tokens=8191, experts=60, topk=6, sequences=37,
             score="sigmoid", dtype="bf16", index="i32", padding=True),
        # a whole batch through the router of the 256-expert layer, 32 packed sequences
        dict(name="balance-whole-batch", op="balance", tokens=131072, experts=256, topk=8,
             sequences=32, score="softmax", dtype="f32", index="i64", padding=True),
        # a small fp32 activation of odd width
        dict(name="checkpoint-odd", op="checkpoint", rows=513, cols=1111, dtype="f32"),
        # the residual stream entering the 256-expert layer (width 7168), one batch
        dict(name="checkpoint-batch", op="checkpoint", rows=32768, cols=7168, dtype="bf16"),
        # a handful of tokens of one expert, fp32, odd width
        dict(name="swiglu-few-tokens", op="swiglu", rows=19, cols=1531, dtype="f32"),
        # the dense model's feed-forward (width 14336), 8192 tokens
        dict(name="swiglu-dense", op="swiglu", rows=8192, cols=14336, dtype="bf16"),
        # eight small experts that share 61 tokens, two of them with none
        dict(name="wgrad-few-tokens", op="wgrad", rows=61, experts=8, out=512, inp=256,
             dy="bf16", grad="f32"),
        # the router's own weight gradient: fp32 logit gradients, 256 rows, many tokens
        dict(name="wgrad-router", op="wgrad", rows=16384, experts=1, out=256, inp=7168,
             dy="f32", grad="f32"),
        # the dense model's key projection
        dict(name="wgrad-dense-k", op="wgrad", rows=8192, experts=1, out=1024, inp=4096,
             dy="bf16", grad="bf16"),
        # 64 experts' up projections, unequal shares of the tokens, some experts idle
        dict(name="wgrad-experts-up", op="wgrad", rows=16384, experts=64, out=2048, inp=7168,
             dy="bf16", grad="bf16"),
        # the dense model's gate projection: the largest product
        dict(name="wgrad-dense-gate", op="wgrad", rows=8192, experts=1, out=14336, inp=4096,
             dy="bf16", grad="bf16"),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "checkpoint", "swiglu", "wgrad", "wgrad"])
    if op == "balance":
        experts = rng.choice([4, 8, 16, 17, 60, 64, 128, 160, 256, 384, 512])
        tokens = _between(rng, 1, min(131072, 131072 * 256 // experts))
        return dict(op=op, tokens=tokens, experts=experts, topk=rng.randint(1, min(8, experts - 2)),
                    sequences=_between(rng, 1, 64), score=rng.choice(["softmax", "sigmoid"]),
                    dtype=rng.choice(["bf16", "f32"]), index=rng.choice(["i32", "i64"]),
                    padding=rng.random() < 0.5)
    if op in ("checkpoint", "swiglu"):
        cols = _between(rng, 1, 16384)
        if rng.random() < 0.6 and cols >= 64:
            cols -= cols % 64
        most = 32768 * 7168 if op == "checkpoint" else 8192 * 14336
        return dict(op=op, rows=_between(rng, 1, min(65536, most // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "f32"]))
    out, inp = _between(rng, 8, 14336), _between(rng, 8, 14336)
    if rng.random() < 0.7:
        out, inp = -(-out // 8) * 8, -(-inp // 8) * 8
    experts = min(_between(rng, 1, 64), max(1, 64 * 2048 * 7168 // (out * inp)))
    dy = rng.choice(["bf16", "bf16", "bf16", "f32"])
    most = 8192 * 14336 * 4096 // (4 if dy == "f32" else 1)
    rows = _between(rng, 1, max(1, min(32768, most // (out * inp))))
    return dict(op=op, rows=rows, experts=experts, out=out, inp=inp, dy=dy,
                grad=rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=g.device, dtype=torch.float32)


def _spans(total, parts, seed, empty):
    """Start of each of `parts` ragged spans of [0, total), and the end of the
    last; with `empty`, about one span in eight holds nothing."""
    g = torch.Generator().manual_seed(seed + 77)
    share = torch.rand(parts, generator=g, dtype=torch.float64) ** 2 + 0.05
    if empty and parts >= 4:
        share[torch.randperm(parts, generator=g)[: parts // 8 + 1]] = 0.0
    ends = torch.round(torch.cumsum(share, 0) / share.sum() * total).long().tolist()
    ends[-1] = total
    return [0] + ends


def _activation(g, rows, cols, dtype):
    """Unit-scale values whose tokens differ in size and with a few outlier channels."""
    x = _normal(g, rows, cols)
    x *= torch.exp(0.3 * _normal(g, rows, 1))
    x *= torch.where(torch.rand(1, cols, generator=g, device=g.device) < 0.005, 15.0, 1.0)
    return x.to(dtype)


def _encode(x):
    """Codes and biased exponents of a checkpoint: the scale of a block is the
    smallest power of two whose 127-fold reaches its largest magnitude."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    xp = torch.zeros(rows, nb * BLOCK, dtype=torch.float32, device=x.device)
    xp[:, :cols] = x
    xb = xp.view(rows, nb, BLOCK)
    m, k = torch.frexp(xb.abs().amax(dim=2))        # amax = m * 2^k, 1/2 <= m < 1
    e = torch.where(m > 127 / 128, k - 6, k - 7)
    e = torch.where(m == 0, torch.full_like(e, -126), e).clamp(min=-126)
    codes = torch.round(torch.ldexp(xb, -e[:, :, None]))
    return codes, e


def _decode(codes, e):
    """Values of codes [rows, blocks, 32] and exponents [rows, blocks]."""
    return torch.ldexp(codes, e[:, :, None]).flatten(1)


def _balance_inputs(case, seed):
    g = torch.Generator(device=_device()).manual_seed(seed)
    T, E, K, S = case["tokens"], case["experts"], case["topk"], case["sequences"]
    logits = 1.5 * _normal(g, T, E) + _normal(g, 1, E)
    if case["padding"] and E - 2 >= K:
        logits[:, torch.randperm(E, generator=g, device=g.device)[:2]] = -math.inf
    logits = logits.to(_DT[case["dtype"]])
    chosen = torch.topk(logits.float(), K, dim=1).indices
    begin = torch.tensor(_spans(T, S, seed, case["padding"]), device=g.device)
    mask = None
    if case["padding"]:
        mask = torch.rand(T, generator=g, device=g.device) > 0.1
        chosen = torch.where(mask[:, None], chosen, torch.full_like(chosen, -1))
    chosen = chosen.to(torch.int64 if case["index"] == "i64" else torch.int32)
    return dict(logits=logits, chosen=chosen, begin=begin.to(torch.int32), mask=mask)


def _wgrad_inputs(case, seed):
    g = torch.Generator(device=_device()).manual_seed(seed)
    T = case["rows"]
    dy = 1e-3 * _normal(g, T, case["out"])
    dy *= torch.exp(0.5 * _normal(g, T, 1))
    codes, e = _encode(_activation(g, T, case["inp"], torch.float32))
    nb = e.shape[1]
    exps = torch.zeros(T, -(-nb // 16) * 16, dtype=torch.uint8, device=g.device)
    exps[:, :nb] = (e + 127).to(torch.uint8)
    spans = _spans(T, case["experts"], seed, True)
    return dict(dy=dy.to(_DT[case["dy"]]), codes=codes.flatten(1).to(torch.int8), exps=exps,
                spans=spans)


def prepare(case, seed):
    dev, op = _device(), case["op"]
    s = dict(case=case)
    if op == "balance":
        s.update(_balance_inputs(case, seed))
        T, E = case["tokens"], case["experts"]
        s.update(loss=torch.empty(1, device=dev),
                 counts=torch.empty(E, dtype=torch.int32, device=dev),
                 load=torch.empty(case["sequences"], E, device=dev),
                 dlogits=torch.empty(T, E, dtype=_DT[case["dtype"]], device=dev))
        if own:   # the workspace that a training program keeps
            m = _package()
            s["ws"] = m.workspace(m.muon_balance_workspace_size(T, E, case["sequences"]), dev)
    elif op in ("checkpoint", "swiglu"):
        g = torch.Generator(device=dev).manual_seed(seed)
        rows, cols, dt = case["rows"], case["cols"], _DT[case["dtype"]]
        names = ("x",) if op == "checkpoint" else ("gate", "up", "dh")
        for n in names:
            s[n] = _activation(g, rows, cols, dt)
        outs = ("back",) if op == "checkpoint" else ("h", "dgate", "dup")
        for n in outs:
            s[n] = torch.empty(rows, cols, dtype=dt, device=dev)
        if op == "swiglu":
            s["h8_values"] = torch.empty(rows, cols, dtype=torch.bfloat16, device=dev)
    else:
        s.update(_wgrad_inputs(case, seed))
        s["offsets"] = torch.tensor(s["spans"], dtype=torch.int32, device=dev)
        s["grad"] = torch.empty(case["experts"], case["out"], case["inp"],
                                dtype=_DT[case["grad"]], device=dev)
        if own:
            m = _package()
            s["ws"] = m.workspace(m.muon_act8_weight_grad_workspace_size(
                case["rows"], case["out"], case["inp"], case["experts"], s["dy"].dtype,
                s["grad"].dtype), dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
COEF = 1e-2


def _plain_balance(s):
    case = s["case"]
    T, E = s["logits"].shape
    K, S = case["topk"], case["sequences"]
    x = s["logits"].float()
    if case["score"] == "softmax":
        top = x.amax(dim=1, keepdim=True)
        a = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
        slope = 1.0
    else:
        a = 1.0 / (1.0 + torch.exp(-x))
        slope = 1.0 - a
    z = a.sum(dim=1, keepdim=True)
    p = torch.where(z > 0, a / z, torch.zeros_like(a))
    on = torch.ones(T, device=x.device) if s["mask"] is None else s["mask"].float()
    p = p * on[:, None]
    seq = torch.searchsorted(s["begin"][1:].contiguous(),
                             torch.arange(T, device=x.device, dtype=torch.int32), right=True)
    n_seq = torch.zeros(S, device=x.device).index_add_(0, seq, on)
    n = n_seq.sum()
    ids = s["chosen"].long()
    taken = (ids >= 0) & (on[:, None] > 0)
    at = (seq[:, None] * E + ids.clamp(min=0)).flatten()
    per_seq = torch.zeros(S * E, dtype=torch.int32, device=x.device)
    per_seq.index_add_(0, at, taken.flatten().to(torch.int32))
    per_seq = per_seq.view(S, E)
    load = E / (K * n_seq.clamp(min=1))[:, None] * per_seq.float()
    psum = torch.zeros(S, E, device=x.device).index_add_(0, seq, p)
    scale = COEF / n.clamp(min=1)
    loss = scale * (load * psum).sum()
    f = load[seq]
    d = scale * p * slope * (f - (f * p).sum(dim=1, keepdim=True))
    return dict(loss=loss.reshape(1), counts=per_seq.sum(dim=0, dtype=torch.int32),
                dlogits=d.to(s["logits"].dtype))


def _plain_swiglu(s):
    dt, cols = s["gate"].dtype, s["gate"].shape[1]
    g, u = s["gate"].float(), s["up"].float()
    h = g * torch.sigmoid(g) * u
    g, u = _decode(*_encode(g))[:, :cols], _decode(*_encode(u))[:, :cols]
    dh, sig = s["dh"].float(), torch.sigmoid(g)
    act = g * sig
    dup = dh * act
    dgate = dh * u * (sig + act * (1.0 - sig))
    again = _decode(*_encode(act * u))[:, :cols]
    return dict(h=h.to(dt), dgate=dgate.to(dt), dup=dup.to(dt), h8_values=again.to(torch.bfloat16))


def _plain_wgrad(s):
    T, inp = s["dy"].shape[0], s["case"]["inp"]
    nb = -(-inp // BLOCK)
    e = s["exps"][:, :nb].to(torch.int32) - 127
    x = _decode(s["codes"].float().view(T, nb, BLOCK), e)[:, :inp]
    dy = s["dy"].float()
    cut = s["spans"]
    return torch.stack([torch.matmul(dy[a:b].T, x[a:b]).to(s["grad"].dtype)
                        for a, b in zip(cut[:-1], cut[1:])])


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "balance":
            return _plain_balance(s)
        if op == "checkpoint":
            x = s["x"]
            return dict(back=_decode(*_encode(x.float()))[:, : x.shape[1]].to(x.dtype))
        if op == "swiglu":
            return _plain_swiglu(s)
        return dict(grad=_plain_wgrad(s))
    m = _package()
    if op == "balance":
        b = m.Balance(s["logits"], s["chosen"], seq_begin=s["begin"], mask=s["mask"],
                      score=s["case"]["score"], coef=COEF)
        m.muon_balance_forward(b, s["loss"], s["counts"], s["load"], s["ws"])
        m.muon_balance_backward(b, s["load"], s["dlogits"])
        return dict(loss=s["loss"], counts=s["counts"], dlogits=s["dlogits"])
    if op == "checkpoint":
        x8 = m.act8_empty(*s["x"].shape, device=s["x"].device)
        m.muon_act8_pack(s["x"], x8)
        m.muon_act8_unpack(x8, s["back"])
        return dict(back=s["back"])
    if op == "swiglu":
        g8, u8, h8 = (m.act8_empty(*s["gate"].shape, device=s["gate"].device) for _ in range(3))
        m.muon_act8_swiglu_forward(s["gate"], s["up"], s["h"], g8, u8)
        m.muon_act8_swiglu_backward(s["dh"], g8, u8, s["dgate"], s["dup"], h8)
        m.muon_act8_unpack(h8, s["h8_values"])
        return dict(h=s["h"], dgate=s["dgate"], dup=s["dup"], h8_values=s["h8_values"])
    x8 = m.Act8(s["codes"], s["exps"], s["case"]["inp"])
    m.muon_act8_weight_grad(s["dy"], x8, s["grad"], s["ws"], offsets=s["offsets"])
    return dict(grad=s["grad"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    size = lambda k: 2 if case[k] == "bf16" else 4
    if case["op"] == "balance":
        # forward and backward are calls of their own in a training step, a model's pass apart:
        # logits are read by each, the gradient is written, the choices are read once
        t, e, b = case["tokens"], case["experts"], size("dtype")
        idx = t * case["topk"] * (4 if case["index"] == "i32" else 8)
        return dict(bytes=3 * t * e * b + idx + 8 * case["sequences"] * e, flops=24 * t * e)
    if case["op"] == "checkpoint":
        # written in the forward pass and read back in the backward pass
        n, b = case["rows"] * case["cols"], size("dtype")
        return dict(bytes=2 * n * b + 2 * n * (1 + 1 / BLOCK), flops=4 * n)
    if case["op"] == "swiglu":
        # forward: gate, up in; h and two checkpoints out.  backward: dh and two checkpoints
        # in; dgate, dup and one checkpoint out, whose values are read back in 16 bits
        n, b = case["rows"] * case["cols"], size("dtype")
        return dict(bytes=6 * n * b + 6 * n * (1 + 1 / BLOCK) + 2 * n, flops=40 * n)
    t, o, i = case["rows"], case["out"], case["inp"]
    return dict(bytes=t * o * size("dy") + t * i * (1 + 1 / BLOCK)
                + case["experts"] * o * i * size("grad"), flops=2 * t * o * i)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_quantised(x):
    """Each value to the nearest multiple (ties to even) of 2^e, e the least integer
    >= -126 with 127 * 2^e >= the largest magnitude among its 32 columns."""
    rows, cols = x.shape
    pad = -cols % BLOCK
    y = torch.nn.functional.pad(x, (0, pad)).reshape(rows, -1, BLOCK)
    big = y.abs().max(dim=2, keepdim=True).values
    e = torch.ceil(torch.log2(torch.clamp(big, min=2.0 ** -126) / 127))
    e = torch.where(127 * torch.exp2(e) < big, e + 1, e)        # the logarithm's own rounding
    e = torch.where(127 * torch.exp2(e - 1) >= big, e - 1, e).clamp(min=-126)
    step = torch.exp2(e)
    return (torch.round(y / step) * step).reshape(rows, -1)[:, :cols]


def _exact_balance(case, seed):
    s = _balance_inputs(case, seed)
    T, E, K = case["tokens"], case["experts"], case["topk"]
    x = s["logits"].double()
    a = x.softmax(dim=1) if case["score"] == "softmax" else x.sigmoid()
    z = a.sum(dim=1, keepdim=True)
    p = a / z
    valid = torch.ones(T, dtype=torch.bool, device=x.device) if s["mask"] is None else s["mask"]
    total = int(valid.sum())
    loss = torch.zeros(1, dtype=torch.float64, device=x.device)
    d = torch.zeros_like(x)
    counts = torch.zeros(E, dtype=torch.int64, device=x.device)
    cut = s["begin"].tolist()
    for lo, hi in zip(cut[:-1], cut[1:]):
        rows = torch.nonzero(valid[lo:hi]).flatten() + lo
        if not len(rows):
            continue
        ids = s["chosen"][rows].long().flatten()
        c = torch.bincount(ids[ids >= 0], minlength=E)
        counts += c
        f = c.double() * E / (K * len(rows))
        q = p[rows]
        loss += COEF / total * (f * q.sum(dim=0)).sum()
        # dL/da_e = (f_e - sum_j f_j p_j) / z, then the score's own derivative
        dp = COEF / total * (f - (q * f).sum(dim=1, keepdim=True))
        if case["score"] == "softmax":
            d[rows] = q * dp
        else:
            d[rows] = dp / z[rows] * a[rows] * (1 - a[rows])
    return dict(loss=loss, counts=counts.to(torch.int32), dlogits=d)


def _exact_swiglu(case, seed):
    s = prepare(case, seed)
    g, u, dh = s["gate"].double(), s["up"].double(), s["dh"].double()
    h = g / (1 + torch.exp(-g)) * u
    g, u = _exact_quantised(g), _exact_quantised(u)
    lam = 1 / (1 + torch.exp(-g))
    return dict(h=h, dgate=dh * u * lam * (1 + g * (1 - lam)), dup=dh * g * lam,
                h8_values=_exact_quantised(g * lam * u))


def _exact_wgrad(case, seed):
    s = _wgrad_inputs(case, seed)
    step = torch.exp2(s["exps"].double() - 127)
    step = step.repeat_interleave(BLOCK, dim=1)[:, : s["codes"].shape[1]]
    x = (s["codes"].double() * step)[:, : case["inp"]]
    dy = s["dy"].double()
    g = torch.empty(case["experts"], case["out"], case["inp"], dtype=torch.float64, device=x.device)
    for i, (a, b) in enumerate(zip(s["spans"][:-1], s["spans"][1:])):
        g[i] = dy[a:b].t() @ x[a:b]
    return dict(grad=g)


def exact(case, seed):
    if case["op"] == "balance":
        return _exact_balance(case, seed)
    if case["op"] == "checkpoint":
        return dict(back=_exact_quantised(prepare(case, seed)["x"].double()))
    if case["op"] == "swiglu":
        return _exact_swiglu(case, seed)
    if 2 * case["rows"] * case["out"] * case["inp"] > 4e12:
        return None
    return _exact_wgrad(case, seed)
