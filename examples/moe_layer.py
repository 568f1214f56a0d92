"""One mixture-of-experts layer over the framework's calls, with 4-bit experts.

Serving: router -> plan -> slot weights -> tokens quantised once and dispatched
as 4-bit records -> gate and up products -> gated activation times the route
weight -> quantised again -> down product -> combine.

Training (the experts' 4-bit weights frozen, the router and the layer's input
trained, as when a 4-bit model is fine-tuned): the same forward pass with the
balance loss and an 8-bit checkpoint of the activation's inputs, then the
gradients of the router's weights and of the hidden states.

    python examples/moe_layer.py            # a small layer, both directions
"""
from __future__ import annotations

import os
import sys
from types import SimpleNamespace

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from combine_moonep_plan_gb300 import Buffer  # noqa: E402


class MoELayer:
    """Router weights [E, H] and 4-bit experts: gate and up [E + R*B, F, H],
    down [E + R*B, H, F]; rows past E are the prefetch slots."""

    def __init__(self, R, S, H, F, E, K, B=None, token_padding=16, scoring="softmax", seed=0):
        kw = dict(S=S, K=K, E=E, num_ep_ranks=R, B=B, token_padding=token_padding)
        self.buf = Buffer(H=H, **kw)
        self.R, self.S, self.H, self.F, self.E, self.K = R, S, H, F, E, K
        self.scoring = scoring
        # a token's record: its codes, its scales, up to whole 16-byte vectors.
        # The second Buffer moves records as rows of bf16-sized elements; plans
        # do not depend on the row length, so both share one.
        self.record = -(-(H // 2 + H // 32) // 16) * 16
        self.buf4 = Buffer(H=self.record // 2, zero_copy_views=False, **kw)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = E + R * self.buf.B
        self.router = torch.randn(E, H, generator=g, device="cuda") * H ** -0.5

        def experts(n, k):
            w = torch.randn(rows, n, k, generator=g, device="cuda").mul_(k ** -0.5)
            return self.buf.quantize_mx(w.bfloat16())

        self.gate, self.up, self.down = experts(F, H), experts(F, H), experts(H, F)

    def forward(self, hidden, balance=0.0, num_tokens=None, training=False):
        """hidden [R, S, H] bf16 -> (out [R, S, H] bf16, what backward reads)."""
        buf, H = self.buf, self.H
        s = SimpleNamespace(hidden=hidden)
        s.logits = hidden.float() @ self.router.T
        s.route = buf.route(s.logits, scoring=self.scoring, balance=balance,
                            num_tokens=num_tokens)
        s.plan = buf.plan(s.route.topk, s.route.tokens_per_expert)
        s.cu = s.plan.cu_seqlens
        weights = (self.gate, self.up, self.down)
        buf.prefetch_weight(s.plan, *(w for w, _ in weights), scales=[x for _, x in weights])
        packed, scales = buf.quantize_mx(hidden)
        tokens = torch.zeros(self.R, self.S, self.record, dtype=torch.uint8, device="cuda")
        tokens[..., :H // 2] = packed
        tokens[..., H // 2:H // 2 + H // 32] = scales
        records, s.weights, _, _ = self.buf4.dispatch(tokens.view(torch.bfloat16),
                                                      s.route.weights, plan=s.plan)
        records = records.view(torch.uint8)
        s.rows = (records[:, :H // 2], records[:, H // 2:H // 2 + H // 32])
        gate = buf.expert_product(s.rows, self.gate, s.cu)
        up = buf.expert_product(s.rows, self.up, s.cu)
        s.act, s.checkpoint = buf.gated_act(gate, up, s.cu, s.weights, checkpoint=training)
        s.act4 = buf.quantize_mx(s.act, cu_seqlens=s.cu)
        s.y = buf.expert_product(s.act4, self.down, s.cu)
        out, _ = buf.combine(s.plan, s.y)
        if not training:
            # a training step keeps the checkpoint, not the activation's inputs
            s.gate, s.up = gate, up
        return out, s

    def _segments(self, cu):
        """(rank, first row, end, weight row) of every used segment."""
        B, NvS = self.buf.B, self.buf.NvS
        for j, ends in enumerate(cu.tolist()):
            start = 0
            for x, end in enumerate(ends):
                if end > start:
                    yield j * NvS + start, j * NvS + end, x if x < self.E else self.E + j * B + x - self.E
                start = end

    def _back_product(self, d, weight, cu, into):
        """Gradient of a product's rows: d [rows, n] times the dequantised
        weights [.., n, k], added into `into` [rows, k] fp32 (the quantisation
        itself passes gradients straight through)."""
        for a, b, w in self._segments(cu):
            into[a:b] += d[a:b].float() @ self.buf.dequantize_mx(
                weight[0][w], weight[1][w], dtype=torch.float32)
        return into

    def backward(self, s, d_out, d_loss=None):
        """d_out [R, S, H] bf16 -> (d_router [E, H], d_hidden [R, S, H] fp32)."""
        buf, n = self.buf, self.R * self.buf.NvS
        d_y, _, _, _ = buf.dispatch(d_out, plan=s.plan)
        zeros = lambda c: torch.zeros(n, c, device="cuda")  # noqa: E731
        s.d_act = self._back_product(d_y, self.down, s.cu, zeros(self.F)).bfloat16()
        s.d_gate, s.d_up, s.d_weights_nvs = buf.gated_act_backward(s.checkpoint, s.d_act, s.cu,
                                                                   s.weights)
        d_rows = self._back_product(s.d_gate, self.gate, s.cu, zeros(self.H))
        s.d_rows = self._back_product(s.d_up, self.up, s.cu, d_rows).bfloat16()
        d_hidden, s.d_weights = buf.combine(s.plan, s.d_rows, s.d_weights_nvs)
        s.d_logits = buf.route_backward(s.route, s.logits, s.d_weights, d_loss)
        d_router = torch.einsum("rse,rsh->eh", s.d_logits, s.hidden.float())
        return d_router, d_hidden.float() + s.d_logits @ self.router


def main():
    layer = MoELayer(R=2, S=64, H=512, F=256, E=8, K=2)
    hidden = torch.randn(2, 64, 512, device="cuda").bfloat16()
    out, _ = layer.forward(hidden)
    print("serving: out", tuple(out.shape), "rms %.3f" % out.float().square().mean().sqrt())
    target = torch.randn_like(hidden)
    for step in range(5):
        out, saved = layer.forward(hidden, balance=0.01, training=True)
        diff = out.float() - target.float()
        d_router, _ = layer.backward(saved, (2 * diff / diff.numel()).bfloat16())
        layer.router -= 0.5 * d_router
        print("step %d: error %.4f balance loss %.5f" %
              (step, diff.square().mean(), saved.route.loss.item()))
    assert layer.buf.get_status() == 0 and layer.buf4.get_status() == 0


if __name__ == "__main__":
    main()
