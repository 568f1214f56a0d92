"""A mixture-of-experts layer whose 4-bit experts are trained.

The layer of moe_layer.py with fp32 parameters behind it: the forward pass runs on
their 4-bit forms (quantisation passes gradients straight through), experts are
picked by score + bias among the best groups, and a step is

    router -> plan -> slot weights -> forward -> backward through the layer
    -> weight gradients over the segments, home experts' and slots'
    -> reduce_grad: the slots' into their home experts'
    -> the gradients' norm -> AdamW with 8-bit moments, into fp32 and bf16
    -> the experts' 4-bit forms anew, and the bias's step

    python examples/moe_train.py            # a few steps of a small layer
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from examples.moe_layer import MoELayer  # noqa: E402


class TrainedMoELayer(MoELayer):
    """MoELayer with trained router and experts; groups and top_groups as
    Buffer.route's."""

    def __init__(self, R, S, H, F, E, K, groups=1, top_groups=1, seed=0, **kw):
        super().__init__(R, S, H, F, E, K, scoring="sigmoid", seed=seed, **kw)
        buf = self.buf
        self.bias = torch.zeros(E, device="cuda")
        self.selection = dict(bias=self.bias, groups=groups, top_groups=top_groups, scale=2.5)
        # fp32 parameters at the 4-bit weights' values, and their bf16 forms
        self.experts = [buf.dequantize_mx(c[:E], s[:E], dtype=torch.float32)
                        for c, s in self._weights()]
        self.bf16 = [w.bfloat16() for w in self.experts]
        self.params = [self.router, *self.experts]
        self.state = buf.adamw_state(self.params, bits=8)
        # the slots' gradients are zero between steps: reduce_grad clears them
        self.grads = [torch.empty_like(w) for w in self.experts]
        self.slots = [torch.zeros(R, buf.B, *w.shape[1:], device="cuda") for w in self.experts]
        self.steps = 0

    def _weights(self):
        return self.gate, self.up, self.down

    def weight_grads(self, s):
        """The experts' gradients of a step that went backward, whole after
        reduce_grad."""
        buf = self.buf
        # what the products read: the 4-bit rows' values
        x, act = (buf.dequantize_mx(*(t.contiguous() for t in rows)) for rows in (s.rows, s.act4))
        for rows, d, grad, slots in ((x, s.d_gate, self.grads[0], self.slots[0]),
                                     (x, s.d_up, self.grads[1], self.slots[1]),
                                     (act, s.d_y, self.grads[2], self.slots[2])):
            buf.expert_weight_grad(rows, d, s.cu, out=(grad, slots))
        buf.reduce_grad(s.plan, self.grads, self.slots)
        return self.grads

    def step(self, hidden, grad_of, lr=1e-3, max_norm=1.0, balance=1e-4):
        """One training step; grad_of(out) gives the output's gradient, bf16.
        Returns (out, saved)."""
        buf, E = self.buf, self.E
        out, s = self.forward(hidden, balance=balance, training=True)
        d_router, _ = self.backward(s, grad_of(out))
        grads = [d_router, *self.weight_grads(s)]
        s.norm = buf.grad_norm(grads)
        self.steps += 1
        buf.adamw(self.params, grads, self.state, lr=lr, step=self.steps, weight_decay=0.0,
                  norm=s.norm, max_norm=max_norm, seed=1, weights=[None, *self.bf16])
        for w, (codes, scales) in zip(self.bf16, self._weights()):
            buf.quantize_mx(w, out=(codes[:E], scales[:E]))
        buf.update_route_bias(self.bias, s.route, 1e-3)
        return out, s


def main():
    layer = TrainedMoELayer(R=2, S=64, H=512, F=256, E=8, K=2, groups=4, top_groups=2)
    hidden = torch.randn(2, 64, 512, device="cuda").bfloat16()
    target = torch.randn_like(hidden)
    for step in range(5):
        out, s = layer.step(hidden, lambda o: (2 * (o.float() - target.float())
                                               / o.numel()).bfloat16())
        print("step %d: error %.4f gradient norm %.3e balance loss %.5f" %
              (step, (out.float() - target.float()).square().mean(), s.norm.item(),
               s.route.loss.item()))
    assert layer.buf.get_status() == 0 and layer.buf4.get_status() == 0


if __name__ == "__main__":
    main()
