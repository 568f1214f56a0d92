"""The router at its edges: long runs of short calls, threads, very small
scores, every form of a row with masks and non-finite logits, and millions of
tokens."""
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


@pytest.mark.parametrize("scope", ["rank", "global"])
def test_loss_repeats_over_many_short_calls(scope):
    """The blocks that add up the loss start at different times; every one of a
    long run of short calls gives the same loss, and the formula's."""
    R, S, E, K = 8, 16, 16, 2
    zn = np.random.default_rng(4).standard_normal((R, S, E)).astype(np.float32)
    z = torch.from_numpy(zn).cuda()
    buf = _buffer(R, S, K, E)
    first = buf.route(z, balance=0.5, scope=scope)
    losses = torch.cat([buf.route(z, balance=0.5, scope=scope).loss for _ in range(500)])
    assert torch.equal(losses, first.loss.expand_as(losses))
    _, _, _, loss, _, _ = ref.route(zn, K, "softmax", [S] * R, 0.5, scope)
    assert abs(first.loss.item() - loss) <= (np.ptp(zn) + S + R * E + 32) * EPS * loss
    assert buf.get_status() == 0


def test_threads_with_contexts_of_different_sizes():
    """The kernel for long rows needs shared memory by its number of experts;
    contexts of different sizes route at the same time, each from a thread."""
    import threading
    failures = []

    def work(E):
        try:
            buf = _buffer(1, 8, 2, E)
            with torch.cuda.stream(torch.cuda.Stream()):
                z = torch.randn(1, 8, E, device="cuda")
                want = buf.route(z).topk
                for _ in range(4000):
                    got = buf.route(z)
                assert torch.equal(got.topk, want)
        except Exception as e:  # noqa: BLE001
            failures.append((E, repr(e)))

    threads = [threading.Thread(target=work, args=(E,)) for E in (4096, 640, 1024)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failures


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("d_loss", [1.0, 1e4, 1e-6])
@pytest.mark.parametrize("E", [8, 24, 48, 128, 200, 300, 500, 640])
def test_gradient_of_very_small_scores(E, d_loss, dtype):
    """Sigmoid scores near 2^-120: their shares are ordinary numbers, and so is
    the gradient.  Bounds as for ordinary scores, the exponential's error that
    of its argument (up to 84, 2^-24 each)."""
    R, S, K = 2, 37, 2
    rng = np.random.default_rng(E)
    z = torch.from_numpy(-83.0 + rng.standard_normal((R, S, E)) * 0.3).to(getattr(torch, dtype))
    zn = z.double().numpy()
    buf = _buffer(R, S, K, E)
    z = z.cuda()
    out = buf.route(z, scoring="sigmoid", balance=0.3)
    ids, w, tpe, loss, coef, _ = ref.route(zn, K, "sigmoid", [S] * R, 0.3, "rank")
    assert np.array_equal(out.topk.cpu().numpy(), ids)
    assert np.all(np.abs(out.weights.cpu().numpy() - w) <= (90 + K + 16) * EPS * w)
    assert abs(out.loss.item() - loss) <= (90 + S + R * E + 32) * EPS * loss
    dw = rng.standard_normal((R, S, K)).astype(np.float32)
    for d in (dw, None):
        dz = buf.route_backward(out, z, None if d is None else torch.from_numpy(d).cuda(),
                                torch.tensor([d_loss], device="cuda"))
        want, mag = ref.route_grad(zn, ids, w, np.zeros_like(dw, np.float64) if d is None
                                   else d.astype(np.float64), coef, d_loss, "sigmoid", [S] * R)
        tol = (3 * 90 + E + K + 48) * EPS * mag
        if dtype == "bfloat16":
            tol = tol + np.abs(want) * 2.0 ** -8
        assert np.all(np.abs(dz.double().cpu().numpy() - want) <= tol)


def _check(buf, z, K, scoring, scope, n, alpha=0.37, d_loss=1.75):
    """Forward and gradient against the 64-bit forms, with the bounds of the
    router's other tests."""
    R, S, E = z.shape
    zn = z.double().cpu().numpy()
    out = buf.route(z, scoring=scoring, balance=alpha, scope=scope, num_tokens=n)
    ids, w, tpe, loss, coef, _ = ref.route(zn, K, scoring, n, alpha, scope)
    assert np.array_equal(out.topk.cpu().numpy(), ids)
    assert np.array_equal(out.tokens_per_expert.cpu().numpy(), tpe)
    fin = zn[np.isfinite(zn) & (zn > -1e30)]
    span = float(min(100.0, np.ptp(fin) if fin.size else 0))
    assert np.all(np.abs(out.weights.cpu().numpy() - w) <= (span + K + 16) * EPS * w + 1e-30)
    assert np.all(np.abs(out.coef.cpu().numpy() - coef) <= 8 * EPS * coef)
    assert abs(out.loss.item() - loss) <= (span + S + R * E + 32) * EPS * loss + 1e-30
    dw = np.random.default_rng(5).standard_normal((R, S, K)).astype(np.float32)
    dz = buf.route_backward(out, z, torch.from_numpy(dw).cuda(),
                            torch.tensor([d_loss], device="cuda"))
    want, mag = ref.route_grad(zn, ids, w, dw.astype(np.float64), coef, d_loss, scoring, n)
    tol = (3 * span + E + K + 48) * EPS * mag + 1e-30
    if z.dtype == torch.bfloat16:
        tol = tol + np.abs(want) * 2.0 ** -8
    assert np.all(np.abs(dz.double().cpu().numpy() - want) <= tol)
    assert buf.get_status() == 0


@pytest.mark.parametrize("kind", ["plain", "ties", "masked"])
@pytest.mark.parametrize("E,K,dtype,scoring", [
    (264, 8, "bfloat16", "softmax"),     # 12 values per lane, whole vectors and not
    (384, 8, "bfloat16", "sigmoid"),
    (301, 6, "float32", "softmax"),
    (383, 32, "bfloat16", "softmax"),
    (65, 32, "float32", "sigmoid"),      # more picks than lanes that hold logits
    (128, 8, "float32", "softmax"),
    (250, 8, "bfloat16", "softmax"),
    (256, 8, "float32", "softmax"),
    (384, 8, "float32", "sigmoid"),
    (512, 16, "float32", "softmax"),
    (640, 8, "bfloat16", "softmax"),     # rows in shared memory
])
def test_warp_forms(E, K, dtype, scoring, kind):
    R, S = 1, 70
    rng = np.random.default_rng(E + K)
    z = rng.standard_normal((R, S, E)) * 2
    if kind == "ties":
        z = np.round(z)
        z[z == 0] *= rng.choice([-1.0, 1.0], size=int((z == 0).sum()))
    elif kind == "masked":               # few logits left, none, only the type's lowest
        z[rng.random(z.shape) < 0.97] = -np.inf
        z[:, 0::7] = -np.inf
        z[:, 1::7] = -3e38
    z = torch.from_numpy(z).to(getattr(torch, dtype)).cuda()
    buf = _buffer(R, S, K, E)
    for n in ([S], [33], [0]):
        for scope in ("rank", "global"):
            _check(buf, z, K, scoring, scope, n)


@pytest.mark.parametrize("E", [128, 256, 384, 512, 640, 4096])
def test_nan_and_infinite_logits(E):
    """Ids stay in range and in order, and other rows are as ever."""
    R, S, K = 1, 24, 8
    z = torch.randn(R, S, E, generator=torch.Generator().manual_seed(E))
    z[0, 3, 7] = float("nan")
    z[0, 4, E - 1] = -float("nan")
    z[0, 5, 9] = float("inf")
    z[0, 6, :] = float("nan")
    z[0, 7, ::2] = float("nan")
    z[0, 8, :] = float("inf")
    bad = np.zeros(S, bool)
    bad[3:9] = True
    buf = _buffer(R, S, K, E)
    for scoring in ("softmax", "sigmoid"):
        out = buf.route(z.cuda(), scoring=scoring)
        assert np.array_equal(out.topk.cpu().numpy(), ref.picks(z.double().numpy(), K))
        _, w, _, _, _, _ = ref.route(z.numpy()[:, ~bad], K, scoring, [int((~bad).sum())], 0.0,
                                     "rank")
        got = out.weights.cpu().numpy()
        span = float(np.ptp(z.numpy()[:, ~bad]))
        assert np.all(np.abs(got[:, ~bad] - w) <= (span + K + 16) * EPS * w)
        assert np.isnan(got[0, [3, 4, 6, 7]]).all()
        if scoring == "sigmoid":         # +inf has a score of one
            assert np.all(np.abs(got[0, 8] - 1 / K) <= 16 * EPS)
        dz = buf.route_backward(out, z.cuda(), torch.ones(R, S, K, device="cuda"))
        assert torch.isfinite(dz[0, torch.from_numpy(~bad)]).all()


def test_loss_of_millions_of_tokens():
    """Probability sums over 4.3 million tokens, 2.2e9 logits: loss,
    coefficients and gradient against sums in 64 bits.  A lane adds one token's
    share at a time, S / (blocks x warps) of them, then the warps', blocks' and
    clusters' sums follow: at most a thousand and a few hundred roundings."""
    S, E, K = 4_300_000, 512, 2
    buf = _buffer(1, S, K, E, B=0, token_padding=1)
    z = torch.empty(S, E, dtype=torch.bfloat16, device="cuda")
    step = 1 << 16
    for i in range(0, S, step):
        z[i:i + step].normal_()
    z = z.view(1, S, E)
    r = buf.route(z, balance=0.01)
    P = torch.zeros(E, dtype=torch.float64, device="cuda")
    for i in range(0, S, step):
        P += torch.softmax(z[0, i:i + step].double(), -1).sum(0)
    c = r.tokens_per_expert[0].double()
    assert int(c.sum()) == S * K
    coef = 0.01 * E * c / (K * float(S) ** 2)
    loss = float((coef * P).sum())
    assert bool(((r.coef[0].double() - coef).abs() <= 8 * EPS * coef).all())
    assert abs(r.loss.item() - loss) <= 1500 * EPS * loss
    d_loss = 3e9                             # the gradient of one of many tokens is small
    dz = buf.route_backward(r, z, None, torch.tensor([d_loss], device="cuda"))
    cn = coef.cpu().numpy()[None]
    for at in (slice(0, 3), slice(S // 2, S // 2 + 3), slice(S - 3, S)):
        zn = z[:, at].double().cpu().numpy()
        want, mag = ref.route_grad(zn, ref.picks(zn, K), np.zeros((1, 3, K)), np.zeros((1, 3, K)),
                                   cn, d_loss, "softmax", [3])
        got = dz[:, at].double().cpu().numpy()
        assert np.all(np.abs(got - want) <= (3 * 12 + E + 48) * EPS * mag
                      + np.abs(want) * 2.0 ** -8)
    assert buf.get_status() == 0
