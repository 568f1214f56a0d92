"""The training operators together, as examples/moe_train.py uses them: a step's
gradients, parameters, moments and bias against plain forms at the step's own
intermediates."""
import numpy as np
import pytest
import torch

from tests import train_refs as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("groups,top_groups,tp", [(1, 1, 16), (4, 2, 1)])
def test_training_steps(groups, top_groups, tp):
    from examples.moe_train import TrainedMoELayer
    R, S, H, F, E, K = 2, 48, 128, 96, 8, 2
    torch.manual_seed(0)
    layer = TrainedMoELayer(R, S, H, F, E, K, groups=groups, top_groups=top_groups,
                            token_padding=tp)
    buf, NvS = layer.buf, layer.buf.NvS
    # a skewed router, so that slots hold experts too
    layer.router.mul_(0.2)
    layer.router[0] += 0.05
    hidden = (torch.randn(R, S, H, device="cuda") + 0.3).bfloat16()
    target = torch.randn(R, S, H, device="cuda")
    for step in range(1, 4):
        before = [t.clone() for t in layer.params]
        bias = layer.bias.clone()
        codes = [t.cpu().numpy() for t in layer.state.tensors]
        m0, v0 = (ref.moment_decode(codes[2 * i], codes[2 * i + 1], i) for i in (0, 1))
        out, s = layer.step(hidden, lambda o: ((o.float() - target) / S).bfloat16(), lr=1e-3)
        # the experts' gradients: home segments and slots of the expert, summed
        cu, copies = s.cu.cpu().numpy(), s.plan.experts_to_copy.cpu().numpy()
        x = _f64(buf.dequantize_mx(*(t.contiguous() for t in s.rows)))
        act = _f64(buf.dequantize_mx(*(t.contiguous() for t in s.act4)))
        assert (copies >= 0).any()
        for rows, d, got in ((x, s.d_gate, layer.grads[0]), (x, s.d_up, layer.grads[1]),
                             (act, s.d_y, layer.grads[2])):
            part, mag = ref.weight_grad(rows, _f64(d), cu, E, R, buf.B, NvS)
            want, size = np.zeros(got.shape), np.zeros(got.shape)
            for w, g in part.items():
                e = w if w < E else copies[(w - E) // buf.B, (w - E) % buf.B]
                want[e] += g
                size[e] += mag[w]
            # sums over at most 2 S K rows, 16 at a time, and of the slots
            tol = (2 * S * K / 16 + 8) * 2.0 ** -22 * size
            assert np.all(np.abs(_f64(got) - want) <= tol)
        assert not any(t.any() for t in layer.slots)
        # the parameters, from the gradients that went in
        d_router = torch.einsum("rse,rsh->eh", s.d_logits, hidden.float())
        grads = [_f64(d_router).reshape(-1)] + [_f64(g).reshape(-1) for g in layer.grads]
        norm = np.sqrt(sum((g ** 2).sum() for g in grads))
        assert abs(s.norm.item() - norm) <= 2.0 ** -18 * norm
        for k, (p, old, g) in enumerate(zip(layer.params, before, grads)):
            o, n = layer.state.offsets[k], layer.state.sizes[k]
            want, _, _ = ref.adamw(_f64(old).reshape(-1), g, m0[o:o + n], v0[o:o + n], step, 1e-3,
                                   0.9, 0.999, 1e-8, 0.0, norm, 1.0)
            # an update is at most some ten times lr; its inputs agree to 2^-17 or, where
            # moment and gradient cancel, to that of their sizes
            assert np.all(np.abs(_f64(p).reshape(-1) - want) <= 2.0 ** -12 * 1e-2 + 2.0 ** -22)
        for w, fp32, (c, sc) in zip(layer.bf16, layer.experts, layer._weights()):
            assert torch.equal(w, fp32.bfloat16())
            want = buf.quantize_mx(w)
            assert torch.equal(c[:E], want[0]) and torch.equal(sc[:E], want[1])
        load = s.route.tokens_per_expert.sum(0)
        want = bias + 1e-3 * torch.sign(load.sum() - load * E).float()
        assert torch.equal(layer.bias, want)
        assert out.isfinite().all()
    assert buf.get_status() == 0 and layer.buf4.get_status() == 0


def test_weight_gradient_against_differences():
    """The loss <c, layer output> with signs of some weights turned: linear in the
    down projection, so its difference is the gradient times the change, but for
    the roundings of y to bf16 (2^-9 relative each) and of the rows combined from
    them (2^-9 of a sum of them), before and after."""
    from examples.moe_train import TrainedMoELayer
    R, S, H, F, E, K = 1, 32, 64, 64, 4, 2
    torch.manual_seed(0)
    layer = TrainedMoELayer(R, S, H, F, E, K)
    buf = layer.buf
    hidden = torch.randn(R, S, H, device="cuda").bfloat16()
    c = torch.randn(R, S, H, device="cuda").bfloat16()
    out, s = layer.forward(hidden, training=True)
    layer.backward(s, c)
    grad = layer.weight_grads(s)[2].clone()
    codes, scales = layer.down
    values = buf.dequantize_mx(codes, scales, dtype=torch.float32)
    c64 = c.double()
    base = (out.double() * c64).sum().item()

    def noise(s):
        used = slice(0, int(s.cu[0, -1]))
        return 2.0 ** -8 * (s.y[used].double().abs() * s.d_y[used].double().abs()).sum().item()

    first = noise(s)
    for e in range(E):
        moved = codes.clone()
        # the codes of four columns of one expert's rows change their sign bits
        moved[e, :, :2] ^= 0x88
        layer.down = (moved, scales)
        changed = buf.dequantize_mx(moved, scales, dtype=torch.float32)
        out2, s2 = layer.forward(hidden, training=True)
        s2.d_y = s.d_y
        layer.down = (codes, scales)
        want = ((changed - values)[e].double() * grad[e].double()).sum().item()
        diff = (out2.double() * c64).sum().item() - base
        assert abs(diff - want) <= first + noise(s2)
    assert buf.get_status() == 0


def test_example_runs():
    from examples import moe_train
    moe_train.main()
