"""Tensors of more than 2^31 elements: the rows at the far end, where an offset
computed in 32 bits would have wrapped, against 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import expert_refs as ref

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _one_expert(rows):
    from combine_moonep_plan_gb300 import Buffer
    buf = Buffer(S=rows, H=32, K=1, E=1, num_ep_ranks=1, B=0, token_padding=1,
                 zero_copy_views=False)
    assert buf.NvS == rows
    return buf, torch.tensor([[rows]], dtype=torch.int32, device="cuda")


def _normal(*shape):
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for i in range(0, shape[0], 1 << 14):
        t[i:i + (1 << 14)].normal_()
    return t


def _np(t):
    return t.double().cpu().numpy()


def test_activation_and_quantisation():
    rows, F = 152_000, 14336                     # 2.18e9 elements
    assert rows * F > 1 << 31
    buf, cu = _one_expert(rows)
    gate, up = _normal(rows, F), _normal(rows, F)
    w = torch.rand(rows, device="cuda")
    act, ckpt = buf.gated_act(gate, up, cu, w, checkpoint=True)
    d = _normal(rows, F)
    dg, du, dw = buf.gated_act_backward(ckpt, d, cu, w)
    packed, scales = buf.quantize_mx(gate, cu_seqlens=cu)
    back = buf.dequantize_mx(packed, scales)
    for at in (slice(0, 2), slice(rows // 2, rows // 2 + 2), slice(rows - 3, rows)):
        g, u, ww, dd = _np(gate[at]), _np(up[at]), _np(w[at])[:, None], _np(d[at])
        want = ref.gated(g, u, ww)
        assert np.all(np.abs(_np(act[at]) - want) <= np.abs(want) * (BF16 + 1e-5) + 1e-38)
        c, s = ref.mx_encode(g, ref.E4M3, 8, 128)
        g8 = ref.mx_decode(c, s, ref.E4M3, 128)
        c, s = ref.mx_encode(u, ref.E4M3, 8, 128)
        u8 = ref.mx_decode(c, s, ref.E4M3, 128)
        wg, wu, wd = ref.gated_grad(g8, u8, ww, dd)
        assert np.all(np.abs(_np(du[at]) - wu) <= np.abs(wu) * (BF16 + 1e-5) + 1e-38)
        sg = ref.sigmoid(g8)
        assert np.all(np.abs(_np(dg[at]) - wg) <= np.abs(wg) * BF16 + 1e-5 * np.abs(
            ww * dd * u8) * sg * (1 + np.abs(g8)) + 1e-38)
        mag = np.abs(dd * g8 * sg * u8).sum(-1)
        assert np.all(np.abs(_np(dw[at]) - wd) <= F * 2.0 ** -23 * mag)
        c, s = ref.mx_encode(g, ref.E2M1, 2, 8)
        assert np.array_equal(scales[at].cpu().numpy(), s)
        assert np.array_equal(_np(back[at]), ref.mx_decode(c, s, ref.E2M1, 8))
    assert buf.get_status() == 0


def test_product():
    rows, N, Kd = 270_000, 8192, 64              # 2.21e9 outputs
    assert rows * N > 1 << 31
    buf, cu = _one_expert(rows)
    a = buf.quantize_mx(_normal(rows, Kd))
    w = buf.quantize_mx(_normal(N, Kd).view(1, N, Kd))
    out = buf.expert_product(a, w, cu)

    def decode(p, s):
        return ref.mx_decode(ref.unpack(p.cpu().numpy()), s.cpu().numpy(), ref.E2M1, 8)

    wv = decode(w[0][0], w[1][0])
    for at in (slice(0, 3), slice(rows // 2, rows // 2 + 3), slice(rows - 5, rows)):
        av = decode(a[0][at], a[1][at])
        want, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
        assert np.all(np.abs(_np(out[at]) - want) <= (Kd // 32 + 2) * 2.0 ** -22 * mag
                      + np.abs(want) * BF16)
    assert buf.get_status() == 0


def test_router():
    rows, E, K = 4_300_000, 512, 2               # 2.2e9 logits
    from combine_moonep_plan_gb300 import Buffer
    buf = Buffer(S=rows, H=8, K=K, E=E, num_ep_ranks=1, B=0, token_padding=1,
                 zero_copy_views=False)
    z = _normal(rows, E).view(1, rows, E)
    r = buf.route(z, balance=0.01)
    dw = torch.ones(1, rows, K, device="cuda")
    dw[..., 1] = -1.0
    dz = buf.route_backward(r, z, dw, torch.zeros(1, device="cuda"))
    for at in (slice(0, 2), slice(rows - 3, rows)):
        zn = _np(z[:, at])
        ids = ref.picks(zn, K)
        assert np.array_equal(r.topk[:, at].cpu().numpy(), ids)
        p = ref.share(ref.scores(zn, "softmax"))
        w = ref.share(np.take_along_axis(p, ids, -1))
        assert np.all(np.abs(_np(r.weights[:, at]) - w) <= 1e-5 * w)
        n = zn.shape[1]
        want, mag = ref.route_grad(zn, ids, w, _np(dw[:, at]), np.zeros((1, E)), 0.0, "softmax",
                                   [n])
        assert np.all(np.abs(_np(dz[:, at]) - want) <= 1e-4 * mag + np.abs(want) * BF16 + 1e-30)
    assert int(r.tokens_per_expert.sum()) == rows * K
    assert buf.get_status() == 0
