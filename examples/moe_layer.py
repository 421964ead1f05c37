"""Trains one mixture-of-experts feed-forward layer with the library's operators.

A router sends every token to its two best of eight gated feed-forward experts.
The tokens are sorted by expert, dispatched to their rows and combined from them
with the router's weights.  The forward pass keeps its activations in 8 bits; the
backward pass rebuilds what it needs from them, forms every weight gradient
straight into the optimizer's gradient buffers, and adds the router's balance
loss.  Muon updates the experts, AdamW the router, both with all gradients
clipped to one norm.  Matrix products between tokens and weights are plain
PyTorch.

    python examples/moe_layer.py [--steps 60] [--tokens 2048]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_02_gb300 as m  # noqa: E402

EXPERTS, TOPK, WIDTH, HIDDEN = 8, 2, 128, 256


class MoeLayer:
    def __init__(self, tokens: int, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rand = lambda *s, scale: scale * torch.randn(*s, generator=g, device=device)
        self.tokens, self.device = tokens, device
        copies = tokens * TOPK
        # weights, gradients and momentum of the experts, one matrix an expert ([out, in])
        self.gate, self.up = (rand(EXPERTS, HIDDEN, WIDTH, scale=WIDTH ** -0.5) for _ in range(2))
        self.down = rand(EXPERTS, WIDTH, HIDDEN, scale=HIDDEN ** -0.5)
        self.router = rand(EXPERTS, WIDTH, scale=WIDTH ** -0.5)
        self.groups, self.grads = [], {}
        for name in ("gate", "up", "down"):
            W = getattr(self, name)
            self.grads[name] = torch.zeros_like(W)
            self.groups.append(m.Group.stacked(W, self.grads[name], torch.zeros_like(W)))
        self.grads["router"] = torch.zeros_like(self.router)
        moments = [torch.zeros_like(self.router) for _ in range(2)]
        self.adamw = m.adamw_groups([self.router], [self.grads["router"]], moments[:1], moments[1:])
        # workspaces live as long as the layer
        size = m.muon_act8_weight_grad_workspace_size
        self.ws_balance = m.workspace(m.muon_balance_workspace_size(tokens, EXPERTS), device)
        self.ws_grad = m.workspace(max(
            size(copies, HIDDEN, WIDTH, EXPERTS, torch.bfloat16, torch.float32),
            size(copies, WIDTH, HIDDEN, EXPERTS, torch.bfloat16, torch.float32),
            size(tokens, EXPERTS, WIDTH, 1, torch.float32, torch.float32)), device)
        self.ws_step = m.workspace(m.muon_step_workspace_size(self.groups), device)
        self.ws_sort = m.workspace(m.muon_moe_sort_workspace_size(tokens, EXPERTS, TOPK), device)
        self.routing = m.Routing.empty(tokens, TOPK, EXPERTS, device)
        self.all_grads = m.Grads(self.groups + self.adamw)
        self.ws_norm = m.workspace(m.muon_grad_norm_workspace_size(self.all_grads), device)
        self.grad_norm, self.grad_scale = torch.empty(1, device=device), torch.empty(1, device=device)
        self.balance_loss = torch.zeros(1, device=device)
        self.counts = torch.zeros(EXPERTS, dtype=torch.int32, device=device)
        self.load = torch.zeros(1, EXPERTS, device=device)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """x [tokens, WIDTH] fp32 -> the layer's output, keeping 8-bit checkpoints."""
        self.logits = x @ self.router.T
        weights, chosen = torch.topk(self.logits.softmax(dim=1), TOPK, dim=1)
        self.balance = m.Balance(self.logits, chosen, coef=1e-2)
        m.muon_balance_forward(self.balance, self.balance_loss, self.counts, self.load, self.ws_balance)
        # the tokens' copies, one expert after the other
        self.chosen, self.weights = chosen, weights
        m.muon_moe_sort(chosen, self.routing, self.ws_sort)
        offsets = self.routing.offsets.tolist()
        self.spans = list(zip(offsets[:-1], offsets[1:]))
        copies = self.tokens * TOPK
        xs = torch.empty(copies, WIDTH, dtype=torch.bfloat16, device=self.device)
        self.x8, self.router_x8 = m.act8_empty(copies, WIDTH), m.act8_empty(self.tokens, WIDTH)
        m.muon_moe_dispatch(x, self.routing, xs, self.x8)
        gate, up = self._project(xs, self.gate), self._project(xs, self.up)
        h = torch.empty_like(gate)
        self.gate8, self.up8 = m.act8_empty(copies, HIDDEN), m.act8_empty(copies, HIDDEN)
        m.muon_act8_pack(x, self.router_x8)
        m.muon_act8_swiglu_forward(gate, up, h, self.gate8, self.up8)
        self.out = self._project(h, self.down)      # of each copy, before its weight
        y = torch.empty_like(x)
        m.muon_moe_combine(self.out, weights, self.routing, y)
        return y

    def backward(self, dy: torch.Tensor) -> torch.Tensor:
        """Gradients of every weight from dy, the gradient of the output; returns that of x."""
        copies = self.out.shape[0]
        dout, dw = torch.empty_like(self.out), torch.empty_like(self.weights)
        m.muon_moe_combine_backward(dy, self.out, self.weights, self.routing, dout, dw)
        dh = self._project(dout, self.down.transpose(1, 2))
        dgate, dup = torch.empty_like(dh), torch.empty_like(dh)
        h8 = m.act8_empty(copies, HIDDEN)
        m.muon_act8_swiglu_backward(dh, self.gate8, self.up8, dgate, dup, h8)
        for group, d, act in zip(self.groups, (dgate, dup, dout), (self.x8, self.x8, h8)):
            m.muon_act8_weight_grad(d, act, group, self.ws_grad, offsets=self.routing.offsets)
        # the router: softmax of the chosen probabilities' gradient, then the balance loss's
        p = self.logits.softmax(dim=1)
        dp = torch.zeros_like(p).scatter_(1, self.chosen, dw)
        dlogits = p * (dp - (p * dp).sum(dim=1, keepdim=True))
        m.muon_balance_backward(self.balance, self.load, dlogits, accumulate=True)
        m.muon_act8_weight_grad(dlogits, self.router_x8, self.grads["router"], self.ws_grad)
        # x: what the experts' projections and the router give back
        dxs = self._project(dgate, self.gate.transpose(1, 2)) + self._project(dup, self.up.transpose(1, 2))
        dx = dlogits @ self.router
        m.muon_moe_dispatch_backward(dxs, self.routing, dx, accumulate=True)
        return dx

    def step(self, t: int, lr: float = 0.02, max_norm: float = 1.0) -> None:
        m.muon_grad_norm(self.all_grads, self.grad_norm, self.grad_scale, self.ws_norm, max_norm=max_norm)
        m.muon_step_batched(self.groups, m.hparams(lr=lr, weight_decay=0.0), self.ws_step,
                            grad_scale=self.grad_scale)
        m.muon_adamw_step(self.adamw, m.adamw_hparams(lr=1e-3, weight_decay=0.0, t=t),
                          grad_scale=self.grad_scale)

    def _project(self, x: torch.Tensor, W: torch.Tensor) -> torch.Tensor:
        y = torch.empty(x.shape[0], W.shape[1], dtype=torch.bfloat16, device=x.device)
        for e, (a, b) in enumerate(self.spans):
            torch.matmul(x[a:b], W[e].T.bfloat16(), out=y[a:b])
        return y


def train(steps: int = 60, tokens: int = 2048, device="cuda", report=print) -> list:
    """Fits a fixed random gated layer; returns the losses."""
    g = torch.Generator(device=device).manual_seed(1)
    teacher = [torch.randn(WIDTH, WIDTH, generator=g, device=device) * WIDTH ** -0.5 for _ in range(2)]
    layer, losses = MoeLayer(tokens, device), []
    for t in range(1, steps + 1):
        x = torch.randn(tokens, WIDTH, generator=g, device=device)
        target = torch.tanh(x @ teacher[0]) @ teacher[1]
        y = layer.forward(x)
        diff = y - target
        losses.append(float(diff.square().mean()))
        layer.backward(2.0 / diff.numel() * diff)
        layer.step(t)
        if t == 1 or t % 10 == 0:
            report(f"step {t}: loss {losses[-1]:.4f}, balance {float(layer.balance_loss):.5f}, "
                   f"gradient norm {float(layer.grad_norm):.3f}, tokens per expert {layer.counts.tolist()}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args()
    train(a.steps, a.tokens)
