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
