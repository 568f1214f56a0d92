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
