"""Plain 64-bit forms of the training operators, written from their formulas in
numpy, and the 8-bit moments' formats."""
import numpy as np

from tests import expert_refs as ref

E4M3 = ref.E4M3
#: codes of the second moment, no sign, five exponent and three mantissa bits
E5M3 = np.array([c / 8 if c < 8 else (1 + c % 8 / 8) * 2.0 ** (c // 8 - 1) for c in range(256)])


def adamw(p, g, m, v, step, lr, b1, b2, eps, wd, norm=None, max_norm=None):
    """(p, m, v) after one step."""
    if norm is not None:
        g = g * min(1.0, max_norm / norm if norm else np.inf)
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    mh, vh = m / (1 - b1 ** step), v / (1 - b2 ** step)
    return p - lr * wd * p - lr * mh / (np.sqrt(vh) + eps), m, v


def moment_decode(codes, scales, second):
    """Values of flat codes [32 n] under scales [n]."""
    if second:
        q = E5M3[codes]
    else:
        q = np.where(codes & 127 == 127, np.nan, E4M3[np.minimum(codes & 127, 126)])
        q = np.where(codes & 128, -q, q)
    f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return (q.reshape(-1, 32) * f[:, None]).reshape(-1)


def moment_scale(x, second):
    """Scale bytes of flat values [32 n]: the least power under which none
    saturates."""
    top = np.abs(x).reshape(-1, 32).max(1)
    most = (E5M3 if second else E4M3)[-1]
    two = np.ldexp(most, np.arange(255) - 127)
    return np.minimum(np.searchsorted(two, top), 254).astype(np.uint8)


def moment_step(x, scales, second):
    """The grid's step at each value, under its block's scale."""
    unit = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32)
    t = np.abs(x) / unit
    low = 0 if second else -6
    e = np.maximum(np.frexp(np.where(t > 0, t, 1e-300))[1] - 1, low)
    return np.ldexp(1.0, e - 3) * unit


def weight_grad(x, d, cu, E, R, B, NvS):
    """{weight row: [N, Kd]} of every segment with rows, and the same of the
    terms' magnitudes."""
    out, mag = {}, {}
    for g, a, n in ref.segments(cu, E, R, B, NvS):
        xs, ds = x[a:a + n].astype(np.float64), d[a:a + n].astype(np.float64)
        out[g] = ds.T @ xs
        mag[g] = np.abs(ds).T @ np.abs(xs)
    return out, mag


def select_values(z, scoring, bias):
    """What selects, in 64 bits: the logits where there is no bias."""
    if bias is None:
        return np.asarray(z, np.float64)
    s = ref.scores(np.asarray(z, np.float64), scoring)
    return (ref.share(s) if scoring == "softmax" else s) + np.asarray(bias, np.float64)


def select(z, K, scoring, bias, groups, top_groups, mode):
    """Picks [R, S, K] in 64 bits."""
    z = np.asarray(z, np.float64)
    R, S, E = z.shape
    c = select_values(z, scoring, bias)
    out = np.zeros(z.shape, bool)
    if top_groups < groups:
        a = ref.scores(z, scoring)
        by = c if bias is not None or mode == "max" else \
            (ref.share(a) if scoring == "softmax" else a)
        parts = -np.sort(-by.reshape(R, S, groups, -1), axis=-1)
        value = parts[..., 0] + (parts[..., 1] if mode == "top2" and E > groups else 0)
        kept = ref.picks(value, top_groups)
        keep = np.zeros((R, S, groups), bool)
        np.put_along_axis(keep, kept, True, -1)
        out = np.repeat(~keep, E // groups, axis=-1)
    # left-out experts behind everything else, by index among equals
    idx = np.broadcast_to(np.arange(E), z.shape)
    key = np.where(np.isnan(c), np.inf, c)
    return np.lexsort((idx, -key, ~np.isnan(c), out), axis=-1)[..., :K]


def select_weights(z, ids, scoring, renormalize, scale, ntok):
    s = ref.scores(np.asarray(z, np.float64), scoring)
    a = ref.share(s) if scoring == "softmax" else s
    ak = np.take_along_axis(a, ids, -1)
    if renormalize:
        if scoring == "softmax":
            # the picks' ratios, also where their shares are far below the rest
            zk = np.take_along_axis(np.asarray(z, np.float64), ids, -1)
            ak = ref.scores(zk, "softmax")
        ak = ref.share(ak)
    live = np.arange(z.shape[1])[None, :] < np.asarray(ntok)[:, None]
    return scale * ak * live[..., None]


def select_grad(z, ids, w, dw, coef, dl, scoring, ntok, renormalize, scale):
    """(gradient, sum of its terms' magnitudes) in 64 bits."""
    z = np.asarray(z, np.float64)
    live = (np.arange(z.shape[1])[None, :] < np.asarray(ntok)[:, None])[..., None]
    p = ref.share(ref.scores(z, scoring))
    c = coef[:, None, :]
    g = dl * p * (c - (p * c).sum(-1, keepdims=True))
    mag = abs(dl) * p * (abs(c) + (p * abs(c)).sum(-1, keepdims=True))
    wd, wm = (w * dw).sum(-1, keepdims=True), (w * abs(dw)).sum(-1, keepdims=True)
    if renormalize:
        t = w * (dw - (wd / scale if scale else 0))
        tm = w * (abs(dw) + (wm / abs(scale) if scale else 0))
    else:
        t, tm = w * dw, w * abs(dw)
        if scoring == "softmax":
            g, mag = g - p * wd, mag + p * wm
    add, addm = np.zeros_like(p), np.zeros_like(p)
    np.put_along_axis(add, ids, t, -1)
    np.put_along_axis(addm, ids, np.abs(tm), -1)
    slope = ref.sigmoid(-z) if scoring == "sigmoid" else 1.0
    return np.where(live, (g + add) * slope, 0), np.where(live, (mag + addm) * slope, 0)
