"""AdamW at the ends of its ranges: the smallest eps, gradients whose squares are
subnormal in fp32, replaced moments.

v = b2 v + (c2 g) g takes three operations, each off by 2^-24 of its result or, below
2^-126, by half of the least subnormal, 2^-150; m takes three of 2^-24.  Between
the two ends that these leave for v the quotient is monotonic, so p is off by no
more than the quotients at the ends, the square root's, the inverse's and the
products' roundings (2^-19 of the update is an upper bound, as for ordinary values),
and its own two.  Where m / (...) is subnormal (a tiny m under a huge eps) its
rounding is 2^-150, 1.25 of that after the rate lr / (1 - b1) = 1.25, and the
rate's product and p's sum add 2^-150 each: below 4 2^-150.  A bf16 p is rounded by
2^-8 of the value before, which may be as large as the larger quotient.
"""
import numpy as np
import pytest
import torch

from tests import train_refs as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B1, B2, LR = 0.9, 0.999, 0.125


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(scope="module")
def buf():
    from combine_moonep_plan_gb300 import Buffer
    return Buffer(S=1, H=8, K=1, E=1, num_ep_ranks=1, zero_copy_views=False)


@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-30, 1e-20, 1e-12, 5.7e-11, 5.8e-11, 1e-8,
                                 2.0 ** 125])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_gradients(buf, eps, bits, dtype):
    """The first step, from gradients of 1e-21 to 1e18 and zeros (32 of a size, a
    block of the 8-bit moments).  Between 5.7e-11 and 5.8e-11, 2^-39 / sqrt(1 - b2),
    8-bit moments change to the root that takes a subnormal v as 0."""
    size = np.repeat(10.0 ** np.arange(-21, 19, 3), 32)
    g = (np.random.default_rng(0).uniform(0.5, 2, size.size) * size).astype(np.float32)
    g[::7] = 0
    p = torch.zeros(g.size, dtype=dtype, device="cuda")
    state = buf.adamw_state([p], bits=bits)
    buf.adamw([p], [torch.from_numpy(g).cuda()], state, lr=LR, step=1, betas=(B1, B2), eps=eps,
              weight_decay=0.0)
    g = g.astype(np.float64)
    want, m, v = ref.adamw(0 * g, g, 0 * g, 0 * g, 1, LR, B1, B2, eps, 0.0)
    dv = 6 * U * v + 3 * 2.0 ** -150
    ends = [np.abs(LR * m / (1 - B1) / (np.sqrt(np.maximum(x, 0) / (1 - B2)) + eps))
            for x in (v - dv, v + dv)]
    tol = ends[0] - ends[1] + 2.0 ** -19 * ends[0] + 4 * 2.0 ** -150
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * ends[0] + 1e-40
    got = p.double().cpu().numpy()
    assert np.all(got[g == 0] == 0)
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("eps", [1e-39, 2.0 ** -126 * (1 - 2.0 ** -23), 2.0 ** 126])
@pytest.mark.parametrize("bits", [32, 8])
def test_eps_out_of_range(buf, eps, bits):
    """An eps that the quotient's inverse cannot take."""
    from combine_moonep_plan_gb300._lib import MoonepError
    p, g = torch.ones(64, device="cuda"), torch.zeros(64, device="cuda")
    state = buf.adamw_state([p], bits=bits)
    with pytest.raises(MoonepError):
        buf.adamw([p], [g], state, lr=1.0, step=1, eps=eps, weight_decay=0.0)
    assert p.eq(1).all()


def test_transposed_gradients_and_copies(buf):
    """Refused, where views of the elements in order are taken."""
    p = [torch.ones(8, 16, device="cuda"), torch.ones(5, device="cuda")]
    g = [torch.ones(16, 8, device="cuda"), torch.ones(5, device="cuda")]
    w = [torch.zeros(16, 8, device="cuda").bfloat16(), None]
    state = buf.adamw_state(p)
    kw = dict(lr=0.5, step=1, weight_decay=0.0)
    with pytest.raises(ValueError):
        buf.adamw(p, g, state, **kw)
    flat = [t.view(-1) for t in g]
    with pytest.raises(ValueError):
        buf.adamw(p, flat, state, weights=w, **kw)
    assert p[0].eq(1).all() and not state.tensors[0].any()
    buf.adamw(p, flat, state, weights=[w[0].view(-1), None], **kw)
    assert (p[0] - 0.5).abs().max().item() < 1e-5 and torch.equal(w[0].view(8, 16), p[0].bfloat16())
    assert (p[1] - 0.5).abs().max().item() < 1e-5
