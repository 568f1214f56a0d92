"""The router on the GPU against its 64-bit form: picks and counts exactly,
weights, loss and gradient within bounds that follow from fp32 arithmetic
(2^-24 per rounding, and an error of |z - max| 2^-24 relative in exp(z - max)).
"""
import numpy as np
import pytest
import torch

from tests import expert_refs as ref

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _buffer(R, S, K, E, **kw):
    from combine_moonep_plan_gb300 import Buffer
    return Buffer(S=S, H=8, K=K, E=E, num_ep_ranks=R, zero_copy_views=False, **kw)


def _logits(R, S, E, kind, seed):
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((R, S, E)) * 2
    if kind == "ties":            # many equal logits, signed zeros
        z = np.round(z)
        z[z == 0] *= rng.choice([-1.0, 1.0], size=int((z == 0).sum()))
    elif kind == "masked":        # -inf and the type's lowest value, some whole rows
        z[rng.random(z.shape) < 0.6] = -np.inf
        z[:, 0::7] = -np.inf
        z[:, 1::7] = -3e38
    elif kind == "large":
        z *= 30
    return torch.from_numpy(z).float()


CASES = [
    # R, S, E, K, scoring, scope, dtype, kind, ntok
    (1, 1, 1, 1, "softmax", "rank", "float32", "plain", None),
    (1, 1, 8, 8, "sigmoid", "global", "float32", "plain", None),
    (2, 64, 8, 2, "softmax", "rank", "float32", "ties", None),
    (2, 5, 8, 3, "softmax", "global", "bfloat16", "ties", [5, 0]),
    (4, 33, 16, 4, "sigmoid", "rank", "bfloat16", "plain", [0, 1, 33, 20]),
    (3, 37, 21, 5, "softmax", "rank", "float32", "masked", [37, 0, 11]),
    (1, 7, 33, 7, "softmax", "global", "float32", "plain", None),
    (8, 17, 64, 6, "sigmoid", "global", "float32", "masked", None),
    (2, 129, 66, 8, "softmax", "rank", "bfloat16", "plain", [129, 64]),
    (8, 16, 128, 8, "softmax", "rank", "float32", "plain", None),
    (8, 100, 256, 8, "sigmoid", "rank", "float32", "plain", [100, 0, 1, 99, 50, 7, 100, 100]),
    (8, 64, 256, 8, "sigmoid", "global", "bfloat16", "large", None),
    (8, 41, 384, 8, "softmax", "global", "float32", "plain", None),
    (1, 50, 500, 32, "sigmoid", "rank", "bfloat16", "ties", None),
    (2, 9, 514, 1, "softmax", "rank", "float32", "plain", None),
    (64, 3, 640, 9, "softmax", "global", "float32", "large", None),
    (1, 40, 4096, 32, "sigmoid", "rank", "float32", "plain", None),
    (1, 3000, 12, 2, "softmax", "rank", "float32", "plain", [2999]),
]


@pytest.mark.parametrize("R,S,E,K,scoring,scope,dtype,kind,ntok", CASES)
def test_route_and_gradient(R, S, E, K, scoring, scope, dtype, kind, ntok):
    z = _logits(R, S, E, kind, seed=R * 1000 + E).to(getattr(torch, dtype)).cuda()
    zn = z.float().cpu().numpy().astype(np.float64)
    n = [S] * R if ntok is None else ntok
    alpha = 0.37
    buf = _buffer(R, S, K, E)
    out = buf.route(z, scoring=scoring, balance=alpha, scope=scope, num_tokens=ntok)
    ids, w, tpe, loss, coef, P = ref.route(zn, K, scoring, n, alpha, scope)
    assert np.array_equal(out.topk.cpu().numpy(), ids)
    assert np.array_equal(out.tokens_per_expert.cpu().numpy(), tpe)
    span = float(min(100.0, np.ptp(zn[np.isfinite(zn) & (zn > -1e30)]) if np.isfinite(zn).any()
                     else 0))
    # below 1e-30 a score may be rounded as a subnormal
    assert np.all(np.abs(out.weights.cpu().numpy() - w) <= (span + K + 16) * EPS * w + 1e-30)
    got = out.coef.cpu().numpy()
    assert np.all(np.abs(got - coef) <= 8 * EPS * coef)
    assert abs(out.loss.item() - loss) <= (span + S + R * E + 32) * EPS * loss + 1e-30
    # gradient, at the GPU's own picks, weights and coefficients
    rng = np.random.default_rng(5)
    dw = torch.from_numpy(rng.standard_normal((R, S, K))).float().cuda()
    dl = torch.tensor([1.75], device="cuda")
    dz = buf.route_backward(out, z, dw, dl)
    assert dz.dtype == z.dtype
    want, mag = ref.route_grad(zn, ids, w, dw.cpu().numpy().astype(np.float64), coef, 1.75,
                               scoring, n)
    tol = (3 * span + E + K + 48) * EPS * mag + 1e-30
    if dtype == "bfloat16":
        tol = tol + np.abs(want) * 2.0 ** -8
    assert np.all(np.abs(dz.float().cpu().numpy() - want) <= tol)
    # the parts alone, and no balance loss at all
    plain = buf.route(z, scoring=scoring, num_tokens=ntok)
    assert plain.loss is None and torch.equal(plain.topk, out.topk)
    assert torch.equal(plain.weights, out.weights)
    assert torch.equal(plain.tokens_per_expert, out.tokens_per_expert)
    only_w = buf.route_backward(plain, z, dw)
    want, mag = ref.route_grad(zn, ids, w, dw.cpu().numpy().astype(np.float64), coef * 0, 0.0,
                               scoring, n)
    tol = (3 * span + E + K + 48) * EPS * mag + 1e-30
    if dtype == "bfloat16":
        tol = tol + np.abs(want) * 2.0 ** -8
    assert np.all(np.abs(only_w.float().cpu().numpy() - want) <= tol)
    only_l = buf.route_backward(out, z)      # d_loss defaults to 1
    want, mag = ref.route_grad(zn, ids, w, np.zeros((R, S, K)), coef, 1.0, scoring, n)
    tol = (3 * span + E + K + 48) * EPS * mag + 1e-30
    if dtype == "bfloat16":
        tol = tol + np.abs(want) * 2.0 ** -8
    assert np.all(np.abs(only_l.float().cpu().numpy() - want) <= tol)
    assert buf.get_status() == 0


@pytest.mark.parametrize("scoring,scope", [("softmax", "rank"), ("sigmoid", "global"),
                                           ("softmax", "global"), ("sigmoid", "rank")])
def test_gradient_against_differences(scoring, scope):
    """Central differences of alpha-loss plus <d_w, w> in 64 bits, the picks
    held fixed: step h = 1e-4 leaves an error near h^2 = 1e-8 of the third
    derivative's size (below the scale of the values) and 1e-12 of rounding."""
    R, S, E, K, n = 2, 6, 12, 3, [6, 4]
    z = _logits(R, S, E, "plain", 9).cuda()
    zn = z.cpu().numpy().astype(np.float64)
    buf = _buffer(R, S, K, E)
    out = buf.route(z, scoring=scoring, balance=2.0, scope=scope, num_tokens=n)
    dw = np.random.default_rng(3).standard_normal((R, S, K))
    dz = buf.route_backward(out, z, torch.from_numpy(dw).float().cuda(),
                            torch.tensor([0.6], device="cuda")).cpu().numpy()
    ids = ref.picks(zn, K)
    dw32 = dw.astype(np.float32).astype(np.float64)

    def value(zz):
        _, w, _, loss, _, _ = ref.route(zz, K, scoring, n, 2.0, scope, ids=ids)
        return 0.6 * loss + (dw32 * w).sum()

    for i in np.ndindex(R, S, E):
        up, dn = zn.copy(), zn.copy()
        up[i] += 1e-4
        dn[i] -= 1e-4
        assert abs((value(up) - value(dn)) / 2e-4 - dz[i]) < 2e-6, i


def test_nan_and_infinite_logits_stay_in_range():
    R, S, E, K = 2, 12, 40, 4
    z = _logits(R, S, E, "plain", 1)
    z[0, 3, 7] = float("nan")
    z[0, 4, 5] = -float("nan")
    z[1, 2, 9] = float("inf")
    z[1, 5, :] = float("nan")
    buf = _buffer(R, S, K, E)
    out = buf.route(z.cuda(), scoring="softmax", balance=1.0)
    ids = out.topk.cpu().numpy()
    zn = z.numpy().astype(np.float64)
    assert np.array_equal(ids, ref.picks(zn, K))
    w = out.weights.cpu().numpy()
    assert np.isnan(w[0, 3]).all() and np.isnan(w[0, 4]).all() and np.isnan(w[1, 5]).all()
    rows = np.ones((R, S), bool)
    rows[0, 3] = rows[0, 4] = rows[1, 2] = rows[1, 5] = False
    assert np.isfinite(w[rows]).all()
    assert out.tokens_per_expert.sum().item() == R * S * K
    dz = buf.route_backward(out, z.cuda(), torch.ones(R, S, K, device="cuda"))
    assert dz.shape == z.shape
    # sigmoid takes +inf as a score of one
    z = _logits(R, S, E, "plain", 1)
    z[1, 2, 9] = float("inf")
    out = buf.route(z.cuda(), scoring="sigmoid")
    _, w, _, _, _, _ = ref.route(z.numpy(), K, "sigmoid", [S] * R, 0.0, "rank")
    assert np.all(np.abs(out.weights.cpu().numpy() - w) <= 64 * EPS * w + 1e-30)


def test_feeds_the_planner_and_repeats_bit_for_bit():
    R, S, E, K = 8, 300, 64, 4
    z = _logits(R, S, E, "plain", 2).cuda()
    buf = _buffer(R, S, K, E)
    n = [300, 0, 17, 299, 300, 300, 1, 128]
    first = buf.route(z, balance=0.01, num_tokens=n)
    plan = buf.plan(first.topk, first.tokens_per_expert)
    assert buf.get_status() == 0
    assert int(plan.cu_seqlens[:, -1].max()) <= buf.NvS
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = buf.route(z, balance=0.01, num_tokens=n)
        dz = buf.route_backward(again, z)
    side.synchronize()
    for f in ("topk", "weights", "tokens_per_expert", "loss", "coef"):
        assert torch.equal(getattr(first, f), getattr(again, f)), f
    assert torch.equal(dz, buf.route_backward(first, z))


def test_no_tokens():
    buf = _buffer(2, 0, 2, 8)
    out = buf.route(torch.empty(2, 0, 8, device="cuda"), balance=1.0)
    assert out.loss.item() == 0 and not out.tokens_per_expert.any() and not out.coef.any()
    assert buf.route_backward(out, torch.empty(2, 0, 8, device="cuda")).numel() == 0
    buf = _buffer(2, 3, 2, 8)
    z = torch.randn(2, 3, 8, device="cuda")
    out = buf.route(z, balance=1.0, scope="global", num_tokens=[0, 0])
    assert out.loss.item() == 0 and not out.coef.any() and not out.weights.any()
    assert out.tokens_per_expert[:, 0].tolist() == [6, 6]
    assert not buf.route_backward(out, z, torch.ones(2, 3, 2, device="cuda")).any()


def test_refusals():
    from combine_moonep_plan_gb300._lib import MoonepError
    buf = _buffer(2, 4, 2, 8)
    z = torch.randn(2, 4, 8, device="cuda")
    with pytest.raises(TypeError):
        buf.route(z.half())
    with pytest.raises(ValueError):
        buf.route(z[:, :3])
    with pytest.raises(ValueError):
        buf.route(z.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        buf.route(z.cpu())
    with pytest.raises(ValueError):
        buf.route(z, scoring="relu")
    with pytest.raises(ValueError):
        buf.route(z, scope="token")
    with pytest.raises(ValueError):
        buf.route(z, num_tokens=[4])
    for bad in ([4, 5], [-1, 4]):
        with pytest.raises(MoonepError):
            buf.route(z, num_tokens=bad)
    out = buf.route(z)
    with pytest.raises(ValueError):
        buf.route_backward(out, z, torch.zeros(2, 4, 3, device="cuda"))
    with pytest.raises(TypeError):
        buf.route_backward(out, z, out=torch.empty_like(z, dtype=torch.bfloat16))
    few = _buffer(1, 4, 3, 2)                 # more picks than experts
    with pytest.raises(MoonepError):
        few.route(torch.randn(1, 4, 2, device="cuda"))
    shifted = torch.randn(2 * 4 * 8 + 1, device="cuda")[1:].view(2, 4, 8)
    with pytest.raises(MoonepError):
        buf.route(shifted)                    # not 16-byte aligned
    buf.destroy()
    with pytest.raises(MoonepError):
        buf.route(z)
