"""The router at its edges: long runs of short calls."""
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
