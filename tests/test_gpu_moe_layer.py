"""The example layer: every step of both directions against 64-bit forms of
the values that the step before it produced, at a real plan with slots, padding
and a short batch."""
import os
import sys

import numpy as np
import pytest
import torch

from tests import expert_refs as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _layer(**kw):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        from moe_layer import MoELayer
    finally:
        sys.path.pop(0)
    return MoELayer(**kw)


def _np(t):
    return t.double().cpu().numpy()


def _decode(pair):
    p, s = (t.cpu().numpy() for t in pair)
    return ref.mx_decode(ref.unpack(p), s, ref.E2M1, 8)


CASES = [dict(R=2, S=33, H=256, F=96, E=8, K=2, token_padding=8, scoring="softmax"),
         dict(R=4, S=16, H=512, F=160, E=16, K=4, token_padding=16, scoring="sigmoid"),
         dict(R=1, S=1, H=64, F=32, E=2, K=1, token_padding=1, scoring="softmax")]


@pytest.mark.parametrize("kw", CASES)
def test_layer_both_directions(kw):
    layer = _layer(**kw)
    R, S, H, F, E, K = (kw[k] for k in ("R", "S", "H", "F", "E", "K"))
    ntok = [max(1, S - 3 * r) for r in range(R)]
    torch.manual_seed(1)
    hidden = torch.randn(R, S, H, device="cuda").bfloat16()
    layer.router[0] += 0.2                       # a hot expert: slots are used
    served, sv = layer.forward(hidden, num_tokens=ntok)
    out, s = layer.forward(hidden, balance=0.05, num_tokens=ntok, training=True)
    assert torch.equal(served, out)
    cu = s.cu.cpu().numpy()
    NvS, B = layer.buf.NvS, layer.buf.B
    segs = ref.segments(cu, E, R, B, NvS)
    if kw["R"] > 1:
        assert any(g >= E for g, _, _ in segs)
    # the router
    ids, w, tpe, loss, coef, _ = ref.route(_np(s.logits), K, kw["scoring"], ntok, 0.05, "rank")
    assert np.array_equal(s.route.topk.cpu().numpy(), ids)
    assert np.array_equal(s.route.tokens_per_expert.cpu().numpy(), tpe)
    assert abs(s.route.loss.item() - loss) <= 1e-5 * loss
    # products, activation, second product, of each segment's own expert
    rows = _decode(s.rows)
    act4 = _decode(s.act4)
    wn = _np(s.weights)
    ex = [_decode(p) for p in (layer.gate, layer.up, layer.down)]
    for g, first, n in segs:
        at = slice(first, first + n)
        for got, wt in ((sv.gate, ex[0]), (sv.up, ex[1])):
            want, mag = rows[at] @ wt[g].T, np.abs(rows[at]) @ np.abs(wt[g]).T
            assert np.all(np.abs(_np(got[at]) - want) <= (H // 32 + 2) * 2.0 ** -22 * mag
                          + np.abs(want) * BF16)
        want = ref.gated(_np(sv.gate[at]), _np(sv.up[at]), wn[at, None])
        assert np.all(np.abs(_np(s.act[at]) - want) <= np.abs(want) * (BF16 + 1e-5) + 1e-38)
        want, mag = act4[at] @ ex[2][g].T, np.abs(act4[at]) @ np.abs(ex[2][g]).T
        assert np.all(np.abs(_np(s.y[at]) - want) <= (F // 32 + 2) * 2.0 ** -22 * mag
                      + np.abs(want) * BF16)
    # the gradients
    d_out = torch.randn(R, S, H, device="cuda").bfloat16()
    d_loss = torch.tensor([0.5], device="cuda")
    d_router, d_hidden = layer.backward(s, d_out, d_loss)
    # rows outside every segment were never written: decode the others only
    used = (np.arange(NvS)[None, :] < cu[:, -1:]).reshape(-1, 1)
    ck = [ref.mx_decode(np.where(used, c.cpu().numpy(), 0), x.cpu().numpy(), ref.E4M3, 128)
          for c, x in ((s.checkpoint[0], s.checkpoint[2]), (s.checkpoint[1], s.checkpoint[3]))]
    d_y, _, _, _ = layer.buf.dispatch(d_out, plan=s.plan)
    dw_nvs = np.zeros(R * NvS)
    for g, first, n in segs:
        at = slice(first, first + n)
        d_act = _np((d_y[at].float() @ torch.from_numpy(ex[2][g]).float().cuda()).bfloat16())
        dg, du, dwv = ref.gated_grad(ck[0][at], ck[1][at], wn[at, None], d_act)
        dw_nvs[at] = dwv
        mag = np.abs(d_act * ck[0][at] * ck[1][at]).sum(-1)
        # d_act is rounded to bf16 from a product summed in another order: one
        # step of bf16 either way
        assert np.all(np.abs(_np(s.d_weights_nvs[at]) - dwv) <= 2 * BF16 * mag + 1e-30)
    dst = s.plan.dst.cpu().numpy().astype(np.int64)
    row = np.where(dst >= 0, dst, -dst - 1).reshape(R, S, K)
    assert np.array_equal(s.d_weights.cpu().numpy(), s.d_weights_nvs.cpu().numpy()[row])
    want, mag = ref.route_grad(_np(s.logits), ids, w, _np(s.d_weights), coef, 0.5,
                               kw["scoring"], ntok)
    assert np.all(np.abs(_np(s.d_logits) - want) <= 2e-5 * mag + 1e-30)
    assert d_router.shape == (E, H) and torch.isfinite(d_router).all()
    assert d_hidden.shape == (R, S, H) and torch.isfinite(d_hidden).all()
    assert layer.buf.get_status() == 0 and layer.buf4.get_status() == 0


def test_serving_replays_as_a_graph():
    """The serving pass allocates from the stream's pool and never asks the
    host, so it captures and replays; the replay equals the eager pass."""
    layer = _layer(R=2, S=32, H=512, F=128, E=8, K=2)
    hidden = torch.randn(2, 32, 512, device="cuda").bfloat16()
    want, _ = layer.forward(hidden)
    plan = layer.buf.new_plan()
    layer.buf.plan = lambda topk, tpe, p=plan, f=layer.buf.plan: f(topk, tpe, plan=p)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.forward(hidden)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _ = layer.forward(hidden)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    hidden.copy_(torch.randn_like(hidden))
    graph.replay()
    torch.cuda.synchronize()
    fresh, _ = layer.forward(hidden)
    torch.cuda.synchronize()
    assert torch.equal(got, fresh)
    assert layer.buf.get_status() == 0


def test_example_runs():
    import subprocess
    res = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "moe_layer.py")],
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    assert res.stdout.count("step") == 5
