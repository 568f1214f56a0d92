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
         "beside none": ([-86.5, -100.0], 16.0), "many": ([-86.9] * 8, 100.0),
         "all lost": ([-90.0, -95.0], 16.0), "largest scale": ([-2.0, -3.0, -2.5], 3.4e38), "negative": ([-85.0, -86.5], -1e6),
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


def _first(v, n):
    """Places of the n largest, a NaN first, equal ones by index."""
    return np.lexsort((np.arange(len(v)), -np.nan_to_num(v, nan=np.inf, posinf=np.inf,
                                                         neginf=-np.inf), ~np.isnan(v)))[:n]


def _select_any(z, bias, scoring, K, groups, top, mode):
    """Picks of rows with any values, from the definition in 64 bits."""
    z = z.astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        if scoring == "sigmoid":
            a = 1 / (1 + np.exp(-z))
        else:
            m = np.where(np.isnan(z), -np.inf, z).max(-1, keepdims=True)
            s = np.where((m == -np.inf) & (z == -np.inf), 0, np.exp(z - m))
            total = s.sum(-1, keepdims=True)
            a = np.where(total == 0, 0, s / np.where(total == 0, 1, total))
        c = z if bias is None else a + bias
        by = a if bias is None and mode == "top2" else c
        out = np.zeros((*z.shape[:-1], K), np.int64)
        size = z.shape[-1] // groups
        for i in np.ndindex(z.shape[:-1]):
            parts = [g[_first(g, 2)] for g in by[i].reshape(groups, size)]
            value = np.array([p.sum() if mode == "top2" else p[0] for p in parts])
            keep = np.sort(_first(value, top))
            ids = (keep[:, None] * size + np.arange(size)).reshape(-1)
            out[i] = ids[_first(c[i][ids], K)]
    return out


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("mode", ["max", "top2"])
@pytest.mark.parametrize("biased", ["no", "finite", "infinite", "nan"])
@pytest.mark.parametrize("E,K,groups,top", [(64, 4, 4, 2), (160, 6, 8, 3), (640, 8, 8, 4),
                                            (120, 5, 40, 9), (64, 4, 1, 1), (60, 7, 12, 5)])
def test_picks_of_rows_that_are_not_finite(scoring, mode, biased, E, K, groups, top):
    """Rows, and biases, with NaNs, infinities and masks: the picks are the
    definition's."""
    S = 12
    rng = np.random.default_rng(E + groups)
    # values far enough apart for 64 bits to order sums the same in any association
    z = (rng.permuted(np.tile(np.arange(E), (1, S, 1)), axis=-1) / E * 6 - 3).astype(np.float32)
    z[0, 0] = -np.inf
    z[0, 1, 7] = np.nan
    z[0, 2, [9, E - 1]] = np.nan
    z[0, 3, 9] = np.inf
    z[0, 4, 1:] = -np.inf
    z[0, 5, [3, E // 2]] = np.inf
    z[0, 6, E // 2:] = -np.inf
    z[0, 7] = np.nan
    z[0, 8, 5], z[0, 8, E - 2] = np.nan, np.inf
    z[0, 9:11] = -np.inf
    z[0, 9, 11], z[0, 10, E - 1] = np.nan, np.nan
    bias = None if biased == "no" else (rng.permutation(E) * 2.0 ** -12).astype(np.float32)
    if biased == "infinite":
        bias[1::4] = -np.inf
        bias[[6, E - 3]] = np.inf
    elif biased == "nan":
        bias[E // 2 + 1] = np.nan
    buf = _buffer(1, S, K, E)
    want = _select_any(z, None if bias is None else bias.astype(np.float64), scoring, K, groups,
                       top, mode)
    for balance in (0.0, 0.5):
        out = buf.route(torch.from_numpy(z).cuda(), scoring=scoring, groups=groups, top_groups=top,
                        group_score=mode, balance=balance, scale=2.0,
                        bias=None if bias is None else torch.from_numpy(bias).cuda())
        got = out.topk.cpu().numpy()
        assert np.array_equal(got, want), [(s, got[0, s], want[0, s]) for s in range(S)
                                           if not np.array_equal(got[0, s], want[0, s])]
    assert out.weights[0, 11].isfinite().all() and buf.get_status() == 0
