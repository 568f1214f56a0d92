"""Plain 64-bit forms of the router, the microscaled formats, the experts'
product and the gated activation, written from their formulas in numpy, and
the layout helpers the tests share."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def nearest(values, a):
    """Index of the nearest of the ascending `values` (ties to the even index:
    both formats number their values consecutively), saturating."""
    hi = np.clip(np.searchsorted(values, a), 0, len(values) - 1)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - values[lo], values[hi] - a
    up = (dhi < dlo) | ((dhi == dlo) & (hi % 2 == 0))
    return np.where(a >= values[-1], len(values) - 1, np.where(up, hi, lo))


def mx_encode(x, values, emax, sign_bit):
    """x [..., cols] float64 -> (codes uint8 [..., cols], scales uint8
    [..., cols/32])."""
    v = np.asarray(x, np.float64).reshape(-1, 32)
    bad = ~np.isfinite(v).all(1)
    v = np.where(bad[:, None], 0, v)
    top = np.abs(v).max(1)
    e = np.where(top > 0, np.frexp(top)[1] - 1 - emax, -127)
    e = np.maximum(e, -127)
    code = nearest(values, np.abs(v) / np.ldexp(1.0, e)[:, None]).astype(np.uint8)
    code |= np.where(np.signbit(v), sign_bit, 0).astype(np.uint8)
    code[bad] = 0
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    return code.reshape(x.shape), s.reshape(*x.shape[:-1], -1)


def mx_decode(codes, scales, values, sign_bit):
    mag = values[codes & (sign_bit - 1)]
    v = np.where(codes & sign_bit, -mag, mag).reshape(*scales.shape, 32)
    f = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return (v * f[..., None]).reshape(codes.shape)


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed):
    return np.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)


def segments(cu, E, R, B, NvS):
    """(group, first row, rows) of every non-empty segment."""
    L = E // R
    out = []
    for g in range(E + R * B):
        j, x = (g // L, g) if g < E else ((g - E) // B, E + (g - E) % B)
        lo, hi = (cu[j, x - 1] if x else 0), cu[j, x]
        if hi > lo:
            out.append((g, j * NvS + int(lo), int(hi - lo)))
    return out


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def scores(z, scoring):
    if scoring == "sigmoid":
        return sigmoid(z)
    m = z.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        return np.where(np.isneginf(m), 0.0, np.exp(z - m))


def share(s):
    t = s.sum(-1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        return np.where(t == 0, 0.0, s / t)


def picks(z, K):
    """Largest first, equal ones by lowest index, NaN first."""
    key = np.where(np.isnan(z), np.inf, z)
    nan = ~np.isnan(z)
    idx = np.broadcast_to(np.arange(z.shape[-1]), z.shape)
    return np.lexsort((idx, -key, nan), axis=-1)[..., :K]


def route(z, K, scoring, ntok, alpha, scope, ids=None):
    """(ids, weights, tokens_per_expert, loss, coef, P) in 64 bits.  `ids`
    fixes the picks (for differences)."""
    z = np.asarray(z, np.float64)
    R, S, E = z.shape
    live = np.arange(S)[None, :] < np.asarray(ntok)[:, None]
    top = picks(z, K) if ids is None else ids
    s = scores(z, scoring)
    w = share(np.take_along_axis(s, top, -1)) * live[..., None]
    p = np.where(live[..., None], share(s), 0)
    cnt = np.zeros((R, E))
    for r in range(R):
        np.add.at(cnt[r], top[r, :ntok[r]].reshape(-1), 1)
    tpe = cnt.copy()
    tpe[:, 0] += (S - np.asarray(ntok)) * K
    P = p.sum(1)
    n = np.asarray(ntok, np.float64)
    coef = np.zeros((R, E))
    if scope == "rank":
        busy = max(1, int((n > 0).sum()))
        for r in range(R):
            if n[r]:
                coef[r] = alpha * E * cnt[r] / (K * n[r]) / n[r] / busy
    elif n.sum():
        coef[:] = alpha * E * cnt.sum(0) / (K * n.sum()) / n.sum()
    out_ids = np.where(live[..., None], top, 0)
    return out_ids, w, tpe, float((coef * P).sum()), coef, P


def route_grad(z, ids, w, dw, coef, dl, scoring, ntok):
    """(gradient, sum of its terms' magnitudes) in 64 bits."""
    z = np.asarray(z, np.float64)
    live = (np.arange(z.shape[1])[None, :] < np.asarray(ntok)[:, None])[..., None]
    p = share(scores(z, scoring))
    c = coef[:, None, :]
    g = dl * p * (c - (p * c).sum(-1, keepdims=True))
    mag = abs(dl) * p * (abs(c) + (p * abs(c)).sum(-1, keepdims=True))
    t = w * (dw - (w * dw).sum(-1, keepdims=True))
    tm = w * (abs(dw) + (w * abs(dw)).sum(-1, keepdims=True))
    add, addm = np.zeros_like(p), np.zeros_like(p)
    np.put_along_axis(add, ids, t, -1)
    np.put_along_axis(addm, ids, tm, -1)
    slope = sigmoid(-z) if scoring == "sigmoid" else 1.0
    return np.where(live, (g + add) * slope, 0), np.where(live, (mag + addm) * slope, 0)


def gated(g, u, w):
    return w * (g * sigmoid(g) * u)


def gated_grad(g, u, w, d):
    s = sigmoid(g)
    return w * d * u * s * (1 + g * (1 - s)), w * d * g * s, (d * g * s * u).sum(-1)
