"""The selecting router where its ways of working meet: the same logits in rows
that one kernel holds in registers and another in 64 bits, rows with a NaN or an
infinity, and scores near the smallest."""
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


def _ranks(z):
    """Each row's values as whole numbers of the same order, a NaN largest."""
    return np.stack([np.unique(r, return_inverse=True)[1] for r in z.reshape(-1, z.shape[-1])]
                    ).reshape(z.shape).astype(np.float64)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,K,groups,top", [(256, 8, 8, 4), (640, 8, 8, 4), (500, 9, 50, 20),
                                            (4096, 6, 4, 1), (40, 4, 40, 7)])
@pytest.mark.parametrize("nan", [False, True])
def test_groups_by_logits(scoring, E, K, groups, top, nan):
    """Without a bias the groups of the largest logits are kept, also where scores
    that differ in their logits are equal in 64 bits (a sigmoid of 38 is 1, a share
    746 below the row's largest logit is 0)."""
    S = 24
    rng = np.random.default_rng(E + K)
    z = rng.uniform(30, 45, (1, S, E)) if scoring == "sigmoid" else rng.uniform(-2e4, 50, (1, S, E))
    z = z.astype(np.float32)
    if nan:
        z[0, ::3, 5] = np.nan
        z[0, 1::3, E - 2] = np.inf
        z[0, 2::3, :E // 2] = -np.inf
    t = torch.from_numpy(z).cuda()
    want = ref.select(_ranks(z), K, "sigmoid", None, groups, top, "max")
    buf = _buffer(1, S, K, E)
    # with the loss's sums and without: both have every score, or none
    for balance in (0.0, 0.5):
        out = buf.route(t, scoring=scoring, groups=groups, top_groups=top, group_score="max",
                        balance=balance)
        assert np.array_equal(out.topk.cpu().numpy(), want)
    assert buf.get_status() == 0


# name: (logits of the picks, scale)
SMALL = {"one": ([-86.5], 16.0), "two": ([-86.0, -87.0], 16.0),
         "beside none": ([-86.5, -100.0], 16.0), "many": ([-86.9] * 8, 100.0), "all lost": ([-90.0, -95.0], 16.0),
         "largest scale": ([-2.0, -3.0, -2.5], 3.4e38), "negative": ([-85.0, -86.5], -1e6),
         "ordinary": ([1.0, 0.5, -0.25], 2.5)}


@pytest.mark.parametrize("E", [32, 700])
@pytest.mark.parametrize("name", sorted(SMALL))
def test_weights_of_small_scores(name, E):
    """Normalised weights are scale times shares, whatever the scores' sum: a score
    below 2^-126 counts as 0, the others' errors are those of exp(|z|), |z| 2^-24
    relative, and a few roundings."""
    picks, scale = SMALL[name]
    K = len(picks)
    z = np.full((1, 3, E), -200.0, np.float32)
    z[..., 3:3 + K] = picks
    buf = _buffer(1, 3, K, E)
    t = torch.from_numpy(z).cuda()
    out = buf.route(t, scoring="sigmoid", scale=scale)
    zn = z.astype(np.float64)
    ids = ref.select(zn, K, "sigmoid", None, 1, 1, "max")
    assert np.array_equal(out.topk.cpu().numpy(), ids)
    s = base.sigmoid(np.take_along_axis(zn, ids, -1))
    s[s < 2.0 ** -126] = 0
    total = s.sum(-1, keepdims=True)
    w = scale * np.divide(s, total, out=np.zeros_like(s), where=total > 0)
    tol = (100 + K + 16) * EPS * np.abs(w)
    assert np.all(np.abs(out.weights.double().cpu().numpy() - w) <= tol)
    dw = np.linspace(-1, 1, 3 * K).reshape(1, 3, K).astype(np.float32)
    dz = buf.route_backward(out, t, torch.from_numpy(dw).cuda()).double().cpu().numpy()
    dw, none = dw.astype(np.float64), np.zeros((1, E))
    want, _ = ref.select_grad(zn, ids, w, dw, none, 0.0, "sigmoid", [3], True, scale)
    # the terms' magnitudes are those of |w| and |scale|: with a negative w the
    # reference's |d_w| + sum w |d_w| / |scale| is a difference, not their sum
    _, mag = ref.select_grad(zn, ids, np.abs(w), dw, none, 0.0, "sigmoid", [3], True, abs(scale))
    assert np.all(np.abs(dz - want) <= (3 * 100 + E + K + 48) * EPS * mag + 1e-30)
