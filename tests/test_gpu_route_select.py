"""The router with a selection bias and groups on the GPU against its 64-bit
form: picks and counts exactly (also where scores lie closer than fp32 tells
apart), weights, loss and gradient within fp32 bounds as in the plain router's
tests (2^-24 per rounding, and an error of |z - max| 2^-24 relative in
exp(z - max))."""
import numpy as np
import pytest
import torch

from tests import expert_refs as base
from tests import train_refs as ref

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


def _inputs(R, S, E, kind, scoring, dtype, seed):
    """(logits tensor, bias or None)."""
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((R, S, E)) * 1.5
    b = np.round(rng.standard_normal(E) * 10) * 1e-3
    if kind == "plain":
        b = None
    elif kind == "ties":       # equal logits under equal biases, often
        z, b = np.round(z), np.round(b, 2)
    elif kind == "masked":     # experts and logits shut out
        z[rng.random(z.shape) < 0.5] = -np.inf
        b[rng.random(E) < 0.2] = -np.inf
    elif kind == "lowest":     # logits at the type's lowest value, whole rows of them
        z[rng.random(z.shape) < 0.7] = -3e38
        z[:, ::5] = -3e38
    elif kind == "shut":       # fewer experts are open than are picked
        b[3:] = -np.inf
    elif kind == "large":      # the bias decides, scores are a rounding beside it
        b = np.round(rng.standard_normal(E)) * 1e4
    t = torch.from_numpy(z).float().to(getattr(torch, dtype))
    if kind == "close":
        # biases that take the first row's values to within their own rounding of
        # one number; the other rows are the first one's with a few logits moved
        zn = t.double().numpy()
        zn[:] = zn[:1, :1]
        s = base.scores(zn[0, 0], scoring)
        b = 0.75 - (base.share(s) if scoring == "softmax" else s)
        move = rng.random(z.shape) < 0.1
        zn = np.where(move, rng.standard_normal(z.shape), zn)
        t = torch.from_numpy(zn).float().to(getattr(torch, dtype))
    return t.cuda(), None if b is None else torch.from_numpy(b).float().cuda()


CASES = [
    # R, S, E, K, groups, top, mode, scoring, renormalize, kind, dtype, ntok
    (1, 1, 1, 1, 1, 1, "max", "sigmoid", True, "bias", "float32", None),
    (2, 9, 8, 2, 4, 2, "top2", "softmax", True, "bias", "float32", [9, 0]),
    (2, 9, 8, 3, 8, 5, "top2", "sigmoid", False, "bias", "bfloat16", None),
    (2, 33, 18, 4, 3, 2, "max", "sigmoid", True, "ties", "float32", None),
    (1, 40, 48, 12, 4, 1, "top2", "sigmoid", True, "bias", "float32", None),
    (4, 21, 64, 6, 8, 4, "top2", "softmax", False, "close", "float32", [21, 0, 1, 7]),
    (2, 50, 100, 8, 5, 2, "max", "softmax", True, "masked", "float32", None),
    (2, 64, 128, 8, 1, 1, "top2", "softmax", True, "bias", "bfloat16", None),
    (5, 33, 160, 6, 8, 3, "max", "softmax", False, "plain", "bfloat16", [33, 2, 0, 32, 9]),
    (5, 33, 160, 6, 8, 3, "top2", "softmax", True, "plain", "float32", None),
    (3, 33, 132, 6, 4, 2, "top2", "sigmoid", True, "close", "float32", None),
    (2, 33, 160, 6, 8, 3, "top2", "sigmoid", True, "ties", "float32", [33, 2]),
    (4, 33, 192, 6, 8, 3, "max", "sigmoid", True, "close", "bfloat16", None),
    (2, 33, 176, 9, 8, 5, "top2", "softmax", True, "masked", "float32", None),
    (8, 64, 256, 8, 8, 4, "top2", "sigmoid", True, "bias", "float32", None),
    (8, 64, 256, 8, 8, 4, "top2", "sigmoid", True, "close", "float32", None),
    (8, 33, 256, 8, 8, 4, "max", "sigmoid", False, "ties", "bfloat16", None),
    (2, 64, 256, 8, 8, 4, "top2", "sigmoid", True, "masked", "float32", [64, 11]),
    (2, 64, 256, 8, 1, 1, "top2", "sigmoid", True, "large", "float32", None),
    (4, 64, 256, 32, 4, 2, "top2", "sigmoid", True, "bias", "float32", None),
    (2, 64, 256, 31, 1, 1, "top2", "softmax", True, "close", "float32", None),
    (8, 41, 384, 8, 1, 1, "max", "sigmoid", True, "close", "bfloat16", None),
    (3, 41, 384, 8, 16, 7, "top2", "sigmoid", True, "bias", "float32", None),
    (2, 33, 96, 5, 4, 2, "top2", "sigmoid", True, "lowest", "float32", None),
    (2, 33, 96, 5, 4, 2, "top2", "softmax", False, "lowest", "bfloat16", [33, 4]),
    (1, 17, 256, 8, 8, 4, "top2", "sigmoid", True, "shut", "float32", None),
    (1, 17, 40, 8, 1, 1, "max", "softmax", True, "shut", "float32", None),
    (1, 17, 700, 8, 7, 2, "max", "sigmoid", False, "shut", "float32", None),
    (1, 50, 500, 9, 50, 20, "top2", "sigmoid", True, "bias", "float32", None),
    (2, 9, 512, 8, 16, 3, "max", "softmax", False, "bias", "float32", None),
    (2, 9, 640, 8, 8, 4, "top2", "sigmoid", True, "close", "float32", [9, 5]),
    (1, 20, 2050, 10, 2, 1, "top2", "softmax", False, "bias", "bfloat16", None),
    (1, 9, 4096, 32, 4096, 40, "top2", "sigmoid", True, "bias", "float32", None),
    (1, 2500, 12, 2, 3, 2, "top2", "sigmoid", True, "bias", "float32", [2499]),
]


@pytest.mark.parametrize("R,S,E,K,groups,top,mode,scoring,renorm,kind,dtype,ntok", CASES)
def test_select_and_gradient(R, S, E, K, groups, top, mode, scoring, renorm, kind, dtype, ntok):
    z, bias = _inputs(R, S, E, kind, scoring, dtype, seed=R * 1000 + E + K)
    zn = z.float().cpu().numpy().astype(np.float64)
    bn = None if bias is None else bias.cpu().numpy().astype(np.float64)
    n = [S] * R if ntok is None else ntok
    scale, alpha = 2.5, 0.37
    buf = _buffer(R, S, K, E)
    kw = dict(scoring=scoring, bias=bias, groups=groups, top_groups=top, group_score=mode,
              renormalize=renorm, scale=scale, num_tokens=ntok)
    out = buf.route(z, balance=alpha, **kw)
    live = np.arange(S)[None, :] < np.asarray(n)[:, None]
    picks = ref.select(zn, K, scoring, bn, groups, top, mode)
    ids = np.where(live[..., None], picks, 0)
    assert np.array_equal(out.topk.cpu().numpy(), ids)
    _, _, tpe, loss, coef, P = base.route(zn, K, scoring, n, alpha, "rank", ids=picks)
    assert np.array_equal(out.tokens_per_expert.cpu().numpy(), tpe)
    w = ref.select_weights(zn, picks, scoring, renorm, scale, n)
    span = float(min(100.0, np.ptp(zn[zn > -1e30])))
    tol = (span + E / 16 + K + 16) * EPS * w + 1e-30
    assert np.all(np.abs(out.weights.cpu().numpy() - w) <= tol)
    assert np.all(np.abs(out.coef.cpu().numpy() - coef) <= 8 * EPS * coef)
    assert abs(out.loss.item() - loss) <= (span + S + R * E + 32) * EPS * loss + 1e-30
    rng = np.random.default_rng(5)
    dw = torch.from_numpy(rng.standard_normal((R, S, K))).float().cuda()
    dl = torch.tensor([1.75], device="cuda")
    for route, c, d, g in ((out, coef, 1.75, dl), (buf.route(z, **kw), coef * 0, 0.0, None)):
        assert torch.equal(route.topk, out.topk) and torch.equal(route.weights, out.weights)
        assert torch.equal(route.tokens_per_expert, out.tokens_per_expert)
        dz = buf.route_backward(route, z, dw, g)
        assert dz.dtype == z.dtype
        want, mag = ref.select_grad(zn, picks, w, dw.cpu().numpy().astype(np.float64), c, d,
                                    scoring, n, renorm, scale)
        tol = (3 * span + E + K + 48) * EPS * mag + 1e-30
        if dtype == "bfloat16":
            tol = tol + np.abs(want) * 2.0 ** -8
        assert np.all(np.abs(dz.float().cpu().numpy() - want) <= tol)
    assert buf.get_status() == 0


def test_long_batches_pick_exactly():
    """Thousands of rows of ordinary logits, some with neighbours closer than
    fp32 tells apart."""
    for E, K, groups, top, dtype in ((256, 8, 8, 4, torch.float32), (384, 8, 1, 1, torch.bfloat16),
                                     (128, 4, 4, 2, torch.bfloat16)):
        R, S = 4, 8192
        g = torch.Generator(device="cuda").manual_seed(E)
        z = torch.randn(R, S, E, generator=g, device="cuda").to(dtype)
        bias = torch.round(torch.randn(E, generator=g, device="cuda") * 10) * 1e-3
        buf = _buffer(R, S, K, E)
        out = buf.route(z, scoring="sigmoid", bias=bias, groups=groups, top_groups=top)
        want = ref.select(z.float().cpu().numpy(), K, "sigmoid", bias.cpu().numpy(), groups, top,
                          "top2")
        assert np.array_equal(out.topk.cpu().numpy(), want)


def test_long_batches_of_shares_pick_exactly():
    """Shares of the row, under biases of their size."""
    for E, K, groups, top, mode in ((160, 6, 8, 3, "top2"), (64, 6, 1, 1, "max"),
                                    (384, 8, 16, 6, "max")):
        R, S = 4, 8192
        g = torch.Generator(device="cuda").manual_seed(E)
        z = torch.randn(R, S, E, generator=g, device="cuda") * 2
        bias = torch.round(torch.randn(E, generator=g, device="cuda") * 10) * (0.1 / E)
        buf = _buffer(R, S, K, E)
        out = buf.route(z, scoring="softmax", bias=bias, groups=groups, top_groups=top,
                        group_score=mode)
        want = ref.select(z.cpu().numpy(), K, "softmax", bias.cpu().numpy(), groups, top, mode)
        assert np.array_equal(out.topk.cpu().numpy(), want)


def test_without_bias_and_groups_it_is_the_plain_router():
    R, S, E, K = 4, 300, 256, 8
    z = torch.randn(R, S, E, device="cuda")
    buf = _buffer(R, S, K, E)
    for scoring in ("softmax", "sigmoid"):
        a = buf.route(z, scoring=scoring, balance=0.1)
        b = buf.route(z, scoring=scoring, balance=0.1, scale=2.0)
        assert torch.equal(a.topk, b.topk) and torch.equal(a.tokens_per_expert, b.tokens_per_expert)
        assert (b.weights - 2 * a.weights).abs().max().item() <= 8 * EPS * 2
        # groups that are all kept leave nothing out
        c = buf.route(z, scoring=scoring, balance=0.1, scale=2.0, groups=8)
        assert torch.equal(b.topk, c.topk) and torch.equal(b.weights, c.weights)


def test_not_finite_logits():
    R, S, E, K = 1, 5, 64, 4
    z = torch.randn(R, S, E, device="cuda")
    z[0, 0] = -float("inf")
    z[0, 1, 7] = float("nan")
    z[0, 2, 9] = float("inf")
    z[0, 3, 1:] = -float("inf")
    bias = torch.arange(E, device="cuda") * 1e-3
    buf = _buffer(R, S, K, E)
    for scoring in ("sigmoid", "softmax"):
        out = buf.route(z, scoring=scoring, bias=bias, groups=4, top_groups=2, balance=0.1)
        ids = out.topk[0].cpu().numpy()
        assert ids.min() >= 0 and ids.max() < E
        assert all(len(set(r)) == K for r in ids.tolist())
        assert out.tokens_per_expert.sum().item() == S * K
        # nothing but the bias tells the first row's experts apart
        assert ids[0].tolist() == [63, 62, 61, 60]
        assert out.weights[0, 0].eq(0).all()
        if scoring == "sigmoid":
            assert ids[1][0] == 7 and out.weights[0, 1].isnan().any()
            assert ids[2][0] == 9 or bias[ids[2][0]] > 0
            assert ids[3][0] in (0, 63)
        assert out.weights[0, 4].isfinite().all()
    assert buf.get_status() == 0


@pytest.mark.parametrize("scoring,renorm", [("softmax", True), ("sigmoid", True),
                                            ("softmax", False), ("sigmoid", False)])
def test_gradient_against_differences(scoring, renorm):
    """Central differences of alpha-loss plus <d_w, w> in 64 bits, the picks
    held fixed: step h = 1e-4 leaves an error near h^2 = 1e-8 of the third
    derivative's size (below ten times the values' scale) and 1e-12 of
    rounding."""
    R, S, E, K, n, scale = 2, 6, 12, 3, [6, 4], 1.5
    z, bias = _inputs(R, S, E, "bias", scoring, "float32", 9)
    zn = z.cpu().numpy().astype(np.float64)
    buf = _buffer(R, S, K, E)
    out = buf.route(z, scoring=scoring, balance=2.0, num_tokens=n, bias=bias, groups=3,
                    top_groups=2, renormalize=renorm, scale=scale)
    dw = np.random.default_rng(3).standard_normal((R, S, K)).astype(np.float32)
    dz = buf.route_backward(out, z, torch.from_numpy(dw).cuda(),
                            torch.tensor([0.6], device="cuda")).cpu().numpy()
    ids = ref.select(zn, K, scoring, bias.cpu().numpy().astype(np.float64), 3, 2, "top2")

    def value(zz):
        _, _, _, loss, _, _ = base.route(zz, K, scoring, n, 2.0, "rank", ids=ids)
        w = ref.select_weights(zz, ids, scoring, renorm, scale, n)
        return 0.6 * loss + (dw.astype(np.float64) * w).sum()

    for i in np.ndindex(R, S, E):
        up, dn = zn.copy(), zn.copy()
        up[i] += 1e-4
        dn[i] -= 1e-4
        assert abs((value(up) - value(dn)) / 2e-4 - dz[i]) <= 1e-6


@pytest.mark.parametrize("R,S,E,K,ntok", [(1, 1, 1, 1, None), (2, 40, 64, 6, [40, 13]),
                                          (3, 7, 21, 2, [0, 0, 0]), (1, 50, 3000, 8, None)])
def test_bias_step(R, S, E, K, ntok):
    z = torch.randn(R, S, E, device="cuda")
    bias = torch.randn(E, device="cuda") * 0.01
    old = bias.clone()
    buf = _buffer(R, S, K, E)
    out = buf.route(z, scoring="sigmoid", bias=bias, num_tokens=ntok)
    assert buf.update_route_bias(bias, out, 0.001) is bias
    n = [S] * R if ntok is None else ntok
    load = np.zeros(E, np.int64)
    for r in range(R):
        np.add.at(load, out.topk[r, :n[r]].cpu().numpy().reshape(-1), 1)
    step = np.sign(sum(n) * K - load * E).astype(np.float32) * np.float32(0.001)
    assert np.array_equal(bias.cpu().numpy(), old.cpu().numpy() + step)
    # a plain route's counts serve as well
    buf.update_route_bias(bias, buf.route(z, num_tokens=ntok), 0.5)
    assert buf.get_status() == 0


def test_bias_balances():
    """Repeated steps even out the loads of skewed logits."""
    R, S, E, K = 2, 1024, 32, 4
    z = torch.randn(R, S, E, device="cuda") + torch.linspace(-1, 1, E, device="cuda")
    buf = _buffer(R, S, K, E)
    bias = torch.zeros(E, device="cuda")
    spread = []
    for _ in range(200):
        out = buf.route(z, scoring="sigmoid", bias=bias, scale=1.5)
        spread.append(out.tokens_per_expert.sum(0).float().std().item())
        buf.update_route_bias(bias, out, 0.005)
    assert min(spread[-5:]) < 0.25 * spread[0]


def test_captured_with_its_bias_step():
    """Replays go on from the bias that the last one left."""
    R, S, E, K = 2, 128, 64, 4
    z = torch.randn(R, S, E, device="cuda") + torch.linspace(-1, 1, E, device="cuda")
    buf = _buffer(R, S, K, E)
    kw = dict(scoring="sigmoid", groups=4, top_groups=2)
    a, b = torch.zeros(E, device="cuda"), torch.zeros(E, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = buf.route(z, bias=a, **kw)
        buf.update_route_bias(a, out, 0.01)
    for _ in range(4):
        graph.replay()
        want = buf.route(z, bias=b, **kw)
        buf.update_route_bias(b, want, 0.01)
        assert torch.equal(out.topk, want.topk) and torch.equal(out.weights, want.weights)
        assert torch.equal(a, b)


@pytest.mark.parametrize("E,groups", [(640, 8), (512, 512), (4096, 4)])
def test_captured_long_rows(E, groups):
    """Rows and groups whose kernels need more shared memory than a launch has by
    itself, first called within a capture."""
    z, bias = _inputs(1, 20, E, "bias", "sigmoid", "float32", E)
    kw = dict(scoring="sigmoid", bias=bias, groups=groups, top_groups=max(2, groups // 2))
    buf = _buffer(1, 20, 4, E)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = buf.route(z, **kw)
    graph.replay()
    want = ref.select(z.cpu().numpy(), 4, "sigmoid", bias.cpu().numpy(), groups,
                      max(2, groups // 2), "top2")
    assert np.array_equal(out.topk.cpu().numpy(), want)


def test_no_tokens_and_no_weight():
    buf = _buffer(2, 0, 2, 8)
    z, bias = torch.zeros(2, 0, 8, device="cuda"), torch.zeros(8, device="cuda")
    out = buf.route(z, bias=bias, balance=0.1)
    assert out.topk.numel() == 0 and not out.tokens_per_expert.any() and out.loss.item() == 0
    assert buf.route_backward(out, z).numel() == 0
    buf.update_route_bias(bias, out, 0.1)
    assert not bias.any()
    # a scale of zero: no weights, no gradient of them
    z, buf = torch.randn(2, 5, 8, device="cuda"), _buffer(2, 5, 2, 8)
    for renorm in (True, False):
        out = buf.route(z, scale=0.0, renormalize=renorm)
        assert out.topk.max() > 0 and not out.weights.any()
        assert not buf.route_backward(out, z, torch.ones_like(out.weights)).any()


def test_few_sms():
    z, bias = _inputs(4, 500, 256, "bias", "sigmoid", "float32", 1)
    kw = dict(scoring="sigmoid", bias=bias, groups=8, top_groups=4, balance=0.1)
    a = _buffer(4, 500, 8, 256).route(z, **kw)
    b = _buffer(4, 500, 8, 256, num_sms=1).route(z, **kw)
    assert torch.equal(a.topk, b.topk) and torch.equal(a.weights, b.weights)
    assert torch.equal(a.tokens_per_expert, b.tokens_per_expert)
    assert abs(a.loss.item() - b.loss.item()) <= 1600 * EPS * a.loss.item()


def test_refusals():
    from combine_moonep_plan_gb300._lib import MoonepError
    buf = _buffer(1, 4, 4, 12)
    z, bias = torch.randn(1, 4, 12, device="cuda"), torch.zeros(12, device="cuda")
    for kw in (dict(groups=5), dict(groups=0), dict(groups=4, top_groups=5),
               dict(groups=4, top_groups=0), dict(groups=4, top_groups=1), dict(top_groups=2),
               dict(groups=2, group_score="mean"), dict(bias=bias[:11]),
               dict(bias=torch.zeros(24, device="cuda")[::2])):
        with pytest.raises(ValueError):
            buf.route(z, **kw)
    with pytest.raises(TypeError):
        buf.route(z, bias=bias.double())
    for scale in (float("nan"), float("inf"), 1e-40, -1e-40):
        with pytest.raises(MoonepError):
            buf.route(z, scale=scale)
    out = buf.route(z, bias=bias)
    with pytest.raises(MoonepError):
        buf.update_route_bias(bias, out, float("nan"))
    with pytest.raises(ValueError):
        _buffer(1, 5, 4, 12).update_route_bias(bias, out, 0.1)
    with pytest.raises(TypeError):
        buf.update_route_bias(bias.half(), out, 0.1)
