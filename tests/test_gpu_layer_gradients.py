"""The example layer's backward pass, step by step against 64-bit forms of the
values that the step before it produced: the experts' row gradients, the gated
activation's, the hidden states' and the router's."""
import numpy as np
import pytest
import torch

from tests import expert_refs as ref
from tests.test_gpu_moe_layer import CASES, _decode, _layer, _np

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8
EPS = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("kw", CASES)
def test_gradients(kw):
    layer = _layer(**kw)
    R, S, H, F, E, K = (kw[k] for k in ("R", "S", "H", "F", "E", "K"))
    ntok = [max(1, S - 3 * r) for r in range(R)]
    torch.manual_seed(2)
    hidden = torch.randn(R, S, H, device="cuda").bfloat16()
    layer.router[0] += 0.2                       # a hot expert: slots are used
    _, s = layer.forward(hidden, balance=0.05, num_tokens=ntok, training=True)
    d_out = torch.randn(R, S, H, device="cuda").bfloat16()
    d_router, d_hidden = layer.backward(s, d_out, torch.tensor([50.0], device="cuda"))
    cu = s.cu.cpu().numpy()
    NvS = layer.buf.NvS
    segs = ref.segments(cu, E, R, layer.buf.B, NvS)
    wn = _np(s.weights)
    gate, up, down = (_decode(p) for p in (layer.gate, layer.up, layer.down))
    used = (np.arange(NvS)[None, :] < cu[:, -1:]).reshape(-1, 1)
    g8, u8 = (ref.mx_decode(np.where(used, c.cpu().numpy(), 0), x.cpu().numpy(), ref.E4M3, 128)
              for c, x in ((s.checkpoint[0], s.checkpoint[2]), (s.checkpoint[1], s.checkpoint[3])))
    d_y, _, _, _ = layer.buf.dispatch(d_out, plan=s.plan)
    covered = np.zeros(R * NvS, bool)
    for g, first, n in segs:
        at = slice(first, first + n)
        covered[at] = True
        # the down product's rows: an fp32 sum of H terms, rounded to bf16
        dy = _np(d_y[at])
        want, mag = dy @ down[g], np.abs(dy) @ np.abs(down[g])
        got = _np(s.d_act[at])
        assert np.all(np.abs(got - want) <= np.abs(want) * BF16 + (H + 2) * EPS * mag)
        # the activation, at the d_act that the layer computed
        dg, du, _ = ref.gated_grad(g8[at], u8[at], wn[at, None], got)
        sg = ref.sigmoid(g8[at])
        tol = np.abs(wn[at, None] * got * u8[at]) * sg * (1 + np.abs(g8[at])) \
            * (np.abs(g8[at]) + 16) * 2 * EPS + np.abs(dg) * BF16 + 1e-38
        assert np.all(np.abs(_np(s.d_gate[at]) - dg) <= tol)
        tol = np.abs(du) * ((np.abs(g8[at]) + 16) * EPS + BF16) + 1e-38
        assert np.all(np.abs(_np(s.d_up[at]) - du) <= tol)
        # the gate and up products' rows
        dg, du = _np(s.d_gate[at]), _np(s.d_up[at])
        want = dg @ gate[g] + du @ up[g]
        mag = np.abs(dg) @ np.abs(gate[g]) + np.abs(du) @ np.abs(up[g])
        assert np.all(np.abs(_np(s.d_rows[at]) - want)
                      <= np.abs(want) * BF16 + (2 * F + 2) * EPS * mag)
    # each token's rows, summed, and the router's part
    dst = s.plan.dst.cpu().numpy().astype(np.int64)
    row = np.where(dst >= 0, dst, -dst - 1).reshape(R, S, K)
    assert covered[row].all()
    rows = _np(s.d_rows)[row]
    total, dz, router = rows.sum(2), _np(s.d_logits), _np(layer.router)
    want = total + dz @ router
    tol = np.abs(total) * BF16 + K * EPS * np.abs(rows).sum(2) \
        + (E + 2) * EPS * (np.abs(dz) @ np.abs(router) + np.abs(total))
    assert np.all(np.abs(_np(d_hidden) - want) <= tol)
    assert np.abs(dz @ router).max() > np.abs(tol).max()     # a term left out would show
    x = _np(hidden)
    want, mag = np.einsum("rse,rsh->eh", dz, x), np.einsum("rse,rsh->eh", np.abs(dz), np.abs(x))
    assert np.all(np.abs(_np(d_router) - want) <= (R * S + 2) * EPS * mag)
    assert np.abs(want).max() > 0
