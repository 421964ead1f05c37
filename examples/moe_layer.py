"""Trains one mixture-of-experts feed-forward layer with the library's operators.

A router sends every token to its two best of eight gated feed-forward experts.
The forward pass keeps its activations in 8 bits; the backward pass rebuilds
what it needs from them, forms every weight gradient straight into the
optimizer's gradient buffers, and adds the router's balance loss; Muon updates
the experts, AdamW the router.  Matrix products between tokens and weights are
plain PyTorch.

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
        flat = chosen.flatten()
        self.order = torch.argsort(flat, stable=True)
        self.source = self.order // TOPK
        self.chosen, self.weights = chosen, weights
        self.offsets = torch.zeros(EXPERTS + 1, dtype=torch.int32, device=self.device)
        self.offsets[1:] = torch.cumsum(self.counts, dim=0)
        self.spans = list(zip(self.offsets[:-1].tolist(), self.offsets[1:].tolist()))
        xs = x[self.source].bfloat16()
        gate, up = self._project(xs, self.gate), self._project(xs, self.up)
        h = torch.empty_like(gate)
        copies = xs.shape[0]
        self.x8, self.router_x8 = m.act8_empty(copies, WIDTH), m.act8_empty(self.tokens, WIDTH)
        self.gate8, self.up8 = m.act8_empty(copies, HIDDEN), m.act8_empty(copies, HIDDEN)
        m.muon_act8_pack(xs, self.x8)
        m.muon_act8_pack(x, self.router_x8)
        m.muon_act8_swiglu_forward(gate, up, h, self.gate8, self.up8)
        self.out = self._project(h, self.down).float()      # of each copy, before its weight
        w = weights.flatten()[self.order]
        return torch.zeros_like(x).index_add_(0, self.source, w[:, None] * self.out)

    def backward(self, dy: torch.Tensor) -> None:
        """Gradients of every weight from dy, the gradient of the output."""
        copies = self.source.numel()
        dout = dy[self.source]
        w = self.weights.flatten()[self.order]
        dw = torch.empty_like(w)
        dw[self.order] = (dout * self.out).sum(dim=1)
        dout = (w[:, None] * dout).bfloat16()
        dh = self._project(dout, self.down.transpose(1, 2))
        dgate, dup = torch.empty_like(dh), torch.empty_like(dh)
        h8 = m.act8_empty(copies, HIDDEN)
        m.muon_act8_swiglu_backward(dh, self.gate8, self.up8, dgate, dup, h8)
        for group, d, act in zip(self.groups, (dgate, dup, dout), (self.x8, self.x8, h8)):
            m.muon_act8_weight_grad(d, act, group, self.ws_grad, offsets=self.offsets)
        # the router: softmax of the chosen probabilities' gradient, then the balance loss's
        p = self.logits.softmax(dim=1)
        dp = torch.zeros_like(p).scatter_(1, self.chosen, dw.view(self.tokens, TOPK))
        dlogits = p * (dp - (p * dp).sum(dim=1, keepdim=True))
        m.muon_balance_backward(self.balance, self.load, dlogits, accumulate=True)
        m.muon_act8_weight_grad(dlogits, self.router_x8, self.grads["router"], self.ws_grad)

    def step(self, t: int, lr: float = 0.02) -> None:
        m.muon_step_batched(self.groups, m.hparams(lr=lr, weight_decay=0.0), self.ws_step)
        m.muon_adamw_step(self.adamw, m.adamw_hparams(lr=1e-3, weight_decay=0.0, t=t))

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
                   f"tokens per expert {layer.counts.tolist()}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args()
    train(a.steps, a.tokens)
