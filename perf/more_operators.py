"""Cases of the experts' training operators, with their plain forms.

Three kinds of case:

  route   the router with a selection bias and expert groups: experts are picked
          by score + bias among the best groups, weighted by score alone; with
          "train" also the balance loss, the logits' gradient and the bias step
  grad    the experts' weight gradients over the plan's segments, into the home
          experts' gradients and the slots' reduce buffers
  step    the gradients' norm and one AdamW step over many tensors, with moments
          in 32 bits or in 8

Rows follow the dispatched layout: R windows of NvS rows, rank j's segments
given by cu_seqlens[j] (padded inclusive ends over E home experts and B slots).

Moments in 8 bits share a power of two per 32 values.  The first moment is E4M3.
The second is an unsigned code of five exponent and three mantissa bits, code c
standing for (c & 7) / 8 below 8 and (1 + (c & 7) / 8) 2^(c / 8 - 1) above.  A
block's power is the smallest for which no value saturates, 2^-127 at least.
Values are rounded to nearest even, or with a seed up with a probability that
makes them right on average, from 16 bits of word(seed, step, tensor, element).
A second moment that is not zero never rounds to zero.
"""
import math

import numpy as np
import torch

own = False

# ---------------------------------------------------------------- the cases


def listed():
    return [
        # one decode step: 16 tokens on each of 8 ranks pick 8 of 256 experts in
        # the best 4 of 8 groups
        dict(name="route decode grouped", kind="route", R=8, S=16, E=256, K=8, groups=8,
             top_groups=4, group_score="top2", scoring="sigmoid", biased=True, renormalize=True,
             scale=2.5, scope="rank", train=False, dtype="float32", ragged=False),
        # a training step's router over the same experts, with its bias step
        dict(name="route train 256 grouped", kind="route", R=8, S=4096, E=256, K=8, groups=8,
             top_groups=4, group_score="top2", scoring="sigmoid", biased=True, renormalize=True,
             scale=2.5, scope="rank", train=True, dtype="float32", ragged=False),
        # probabilities kept as they are, groups by their best expert, an odd
        # group size, bf16 logits and unequal token counts
        dict(name="route train 160 softmax", kind="route", R=5, S=3001, E=160, K=6, groups=8,
             top_groups=3, group_score="max", scoring="softmax", biased=False, renormalize=False,
             scale=16.0, scope="global", train=True, dtype="bfloat16", ragged=True),
        # 384 experts without groups, a long batch
        dict(name="route train 384 biased", kind="route", R=8, S=8192, E=384, K=8, groups=1,
             top_groups=1, group_score="top2", scoring="sigmoid", biased=True, renormalize=True,
             scale=2.827, scope="rank", train=True, dtype="bfloat16", ragged=False),
        # few rows per expert: the outputs' bytes are all there is
        dict(name="grad few rows", kind="grad", R=2, E=16, B=4, C=512, tp=16, N=1536, Kd=4096,
             skew=1.0, accumulate=False),
        # odd sizes without padding, added to gradients of an earlier batch
        dict(name="grad ragged odd", kind="grad", R=3, E=21, B=4, C=1237, tp=1, N=1000, Kd=1184,
             skew=1.2, accumulate=True),
        # a training step of a 64-expert layer, up projection
        dict(name="grad 64 experts up", kind="grad", R=8, E=64, B=8, C=16384, tp=128, N=2048,
             Kd=7168, skew=0.5, accumulate=False),
        # its down projection on a share of the ranks, a second micro-batch
        dict(name="grad 32 experts down", kind="grad", R=4, E=32, B=8, C=8192, tp=128, N=7168,
             Kd=2048, skew=0.8, accumulate=True),
        # the router and a few vectors beside the experts
        dict(name="step small", kind="step", layout="even", tensors=6, elements=300000,
             dtype="float32", grad="float32", bits=32, seeded=False, clip=True, copy=False),
        # many odd tensors of a model held in bf16 alone
        dict(name="step many odd", kind="step", layout="odd", tensors=160, elements=40000000,
             dtype="bfloat16", grad="bfloat16", bits=8, seeded=True, clip=False, copy=False),
        # one layer's experts: fp32 parameters and moments, and the bf16 weights
        dict(name="step experts", kind="step", layout="even", tensors=3, elements=704643072,
             dtype="float32", grad="float32", bits=32, seeded=False, clip=True, copy=True),
        # the same with moments in 8 bits
        dict(name="step experts 8 bits", kind="step", layout="even", tensors=3,
             elements=704643072, dtype="float32", grad="float32", bits=8, seeded=True, clip=True,
             copy=True),
    ]


def _log(rng, lo, hi, mult=1):
    """A multiple of `mult` in [lo, hi], spread over the logarithm."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / mult)) * mult
        if lo <= v <= hi:
            return v


def draw(rng):
    kind = rng.choice(["route", "grad", "step"])
    if kind == "route":
        R = rng.choice([1, 2, 4, 5, 8])
        groups = rng.choice([1, 1, 2, 3, 4, 8, 16])
        lcm = R * groups // math.gcd(R, groups)
        E = lcm * max(1, _log(rng, 8, 512) // lcm)
        top_groups = rng.randint(1, groups)
        return dict(kind=kind, R=R, S=_log(rng, 1, 65536 // R), E=E,
                    K=rng.randint(1, min(8, E // groups * top_groups)), groups=groups,
                    top_groups=top_groups, group_score=rng.choice(["top2", "max"]),
                    scoring=rng.choice(["softmax", "sigmoid"]), biased=rng.random() < 0.7,
                    renormalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5, 16.0]),
                    scope=rng.choice(["rank", "global"]), train=rng.random() < 0.7,
                    dtype=rng.choice(["float32", "bfloat16"]), ragged=rng.random() < 0.5)
    if kind == "grad":
        while True:
            R = rng.choice([1, 2, 4, 8])
            E = R * _log(rng, 1, 128 // R)
            B = rng.randint(0, E // R)
            c = dict(kind=kind, R=R, E=E, B=B, C=_log(rng, 8, 131072 // R),
                     tp=rng.choice([1, 8, 16, 128]), N=_log(rng, 128, 7168, 8),
                     Kd=_log(rng, 128, 7168, 8), skew=rng.choice([0.0, 0.5, 1.0]),
                     accumulate=rng.random() < 0.4)
            if (E + R * B) * c["N"] * c["Kd"] <= 1800000000 and \
                    R * c["C"] * c["N"] * c["Kd"] <= 131072 * 2048 * 7168:
                return c
    dtype = rng.choice(["float32", "float32", "bfloat16"])
    return dict(kind=kind, layout=rng.choice(["odd", "even"]), tensors=_log(rng, 1, 300),
                elements=_log(rng, 20000, 500000000), dtype=dtype,
                grad=rng.choice(["float32", "bfloat16"]), bits=rng.choice([32, 8]),
                seeded=rng.random() < 0.5, clip=rng.random() < 0.5,
                copy=dtype == "float32" and rng.random() < 0.5)


# ------------------------------------------------------------------- inputs


def _segments(c, seed):
    """cu_seqlens [R, E+B] of a balanced plan: every rank holds C routes over
    its E/R home experts and some of its B slots, each segment padded to tp;
    also the row capacity and the used segments as (rank, start, end, weight
    row)."""
    rng = np.random.Generator(np.random.PCG64(seed))
    R, E, B, C, tp = c["R"], c["E"], c["B"], c["C"], c["tp"]
    L = E // R
    nvs = -(-(C + (L + B) * (tp - 1)) // tp) * tp
    cu = np.zeros((R, E + B), np.int32)
    segs = []
    for j in range(R):
        slots = int(rng.integers(0, B + 1)) if B else 0
        p = (1.0 + rng.permutation(L + slots)) ** -c["skew"]
        n = rng.multinomial(C, p / p.sum())
        size = np.zeros(E + B, np.int64)
        size[j * L:(j + 1) * L] = n[:L]
        size[E:E + slots] = n[L:]
        size = -(-size // tp) * tp
        end = np.cumsum(size)
        cu[j] = end
        for x in np.nonzero(size)[0]:
            w = int(x) if x < E else E + j * B + int(x) - E
            segs.append((j, int(end[x] - size[x]), int(end[x]), w))
    return cu, nvs, segs


def _sizes(c):
    """Sizes of a step's tensors and their first elements in one storage, each
    on a multiple of 32."""
    n, total = c["tensors"], c["elements"]
    if c["layout"] == "even":
        each = max(1, total // n)
        sizes = [each] * n
    else:
        # a geometric spread over three decades, every size odd
        share = [10 ** (3 * ((i * 37) % n) / n) for i in range(n)]
        sizes = [max(1, int(total * s / sum(share))) | 1 for s in share]
    first = np.concatenate([[0], np.cumsum([-(-s // 32) * 32 for s in sizes])])
    return sizes, [int(v) for v in first]


_HYPER = dict(lr=1e-4, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)
_STEP, _SEED, _MAX_NORM = 1000, 77, 1.0


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = c["kind"]

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)

    st = dict(c)
    if kind == "route":
        R, S, E = c["R"], c["S"], c["E"]
        popular = normal(E, dtype=torch.float32, std=0.5)
        z = normal(R, S, E, dtype=torch.float32).add_(popular)
        st["logits"] = z.to(getattr(torch, c["dtype"]))
        # whole steps of the bias rate against the popular experts
        st["bias"] = (torch.round(normal(E, dtype=torch.float32, std=8) - 40 * popular) * 1e-3
                      if c["biased"] else None)
        rng = np.random.Generator(np.random.PCG64(seed))
        st["num_tokens"] = [int(rng.integers(0, S + 1)) for _ in range(R)] if c["ragged"] \
            else [S] * R
        st["d_weights"] = normal(R, S, c["K"], dtype=torch.float32, std=1e-3)
        st["d_loss"] = torch.full((1,), 0.5, device="cuda")
        if own:
            from combine_moonep_plan_gb300 import Buffer
            st["buffer"] = Buffer(S=S, H=8, K=c["K"], E=E, num_ep_ranks=R,
                                  zero_copy_views=False)
        return st
    if kind == "grad":
        cu, nvs, segs = _segments(c, seed)
        st["cu_seqlens"], st["segments"] = torch.from_numpy(cu).cuda(), segs
        st["NvS"] = nvs
        R, E, B, N, Kd = c["R"], c["E"], c["B"], c["N"], c["Kd"]
        st["x"], st["d"] = normal(R * nvs, Kd), normal(R * nvs, N, std=1e-2)
        st["grad"] = torch.zeros(E, N, Kd, device="cuda")
        st["slots"] = torch.zeros(R, B, N, Kd, device="cuda")
        if c["accumulate"]:
            st["grad"].normal_(generator=g).mul_(0.1)
        if own:
            from combine_moonep_plan_gb300 import Buffer
            st["buffer"] = Buffer(S=c["C"], H=8, K=1, E=E, num_ep_ranks=R, B=B,
                                  token_padding=c["tp"], zero_copy_views=False)
        return st
    sizes, first = _sizes(c)
    n = first[-1]
    live = torch.zeros(n, dtype=torch.bool, device="cuda")
    for a, s in zip(first, sizes):
        live[a:a + s] = True
    views = lambda t: [t[a:a + s] for a, s in zip(first, sizes)]  # noqa: E731
    st["first"] = torch.tensor(first[:-1], device="cuda")
    st["p"] = normal(n, dtype=torch.float32, std=0.02).mul_(live).to(getattr(torch, c["dtype"]))
    # gradients of tensors and elements of differing size
    size = torch.exp(normal(n // 32, 1, dtype=torch.float32)).expand(-1, 32).reshape(-1) * 1e-3
    st["g"] = normal(n, dtype=torch.float32).mul_(size).mul_(live).to(getattr(torch, c["grad"]))
    m = normal(n, dtype=torch.float32, std=0.3).mul_(size).mul_(live)
    v = normal(n, dtype=torch.float32).square_().mul_(0.5).add_(0.5).mul_(size).mul_(size)
    v = v.mul_(live)
    if c["bits"] == 8:
        m8, ms = _encode_m(m, None)
        v8, vs = _encode_v(v, None)
        st["moments"] = (m8, ms, v8, vs)
    else:
        st["moments"] = (m, v)
    st["copy"] = torch.zeros(n, dtype=torch.bfloat16, device="cuda") if c["copy"] else None
    st["params"], st["grads"] = views(st["p"]), views(st["g"])
    st["weights"] = views(st["copy"]) if c["copy"] else None
    if own:
        from combine_moonep_plan_gb300 import Buffer
        st["buffer"] = Buffer(S=1, H=8, K=1, E=1, num_ep_ranks=1, zero_copy_views=False)
        st["state"] = st["buffer"].adamw_state(st["params"], bits=c["bits"])
        for to, have in zip(st["state"].tensors, st["moments"]):
            to.copy_(have)
    return st


# ---------------------------------------------------------------- the passes


def run(state):
    return _calls(state) if own else _plain(state)


def _calls(st):
    """What a user of the framework writes."""
    buf, kind = st["buffer"], st["kind"]
    if kind == "route":
        r = buf.route(st["logits"], scoring=st["scoring"], balance=1e-4 if st["train"] else 0.0,
                      scope=st["scope"], num_tokens=st["num_tokens"], bias=st["bias"],
                      groups=st["groups"], top_groups=st["top_groups"],
                      group_score=st["group_score"], renormalize=st["renormalize"],
                      scale=st["scale"])
        out = dict(topk=r.topk, weights=r.weights, tokens_per_expert=r.tokens_per_expert)
        if st["train"]:
            out["loss"] = r.loss
            out["d_logits"] = buf.route_backward(r, st["logits"], st["d_weights"], st["d_loss"])
            if st["biased"]:
                out["bias"] = buf.update_route_bias(st["bias"], r, 1e-3)
        return out
    if kind == "grad":
        grad, slots = buf.expert_weight_grad(st["x"], st["d"], st["cu_seqlens"],
                                             out=(st["grad"], st["slots"]),
                                             accumulate=st["accumulate"])
        return dict(grad=grad, slots=slots)
    out = {}
    if st["clip"]:
        out["norm"] = buf.grad_norm(st["grads"])
    buf.adamw(st["params"], st["grads"], st["state"], step=_STEP, **_HYPER,
              norm=out.get("norm"), max_norm=_MAX_NORM if st["clip"] else None,
              seed=_SEED if st["seeded"] else None, weights=st["weights"])
    out["p"] = st["p"]
    out["m"], out["v"] = st["state"].moments()
    if st["copy"] is not None:
        out["copy"] = st["copy"]
    return out


def _plain(st):
    kind = st["kind"]
    if kind == "route":
        return _plain_route(st)
    if kind == "grad":
        # one product for each used segment: there is no elementary operation
        # over ragged groups
        x, d, nvs, E = st["x"], st["d"], st["NvS"], st["E"]
        flat = st["slots"].view(-1, st["N"], st["Kd"])
        if not st["accumulate"]:
            st["grad"].zero_()
        for j, a, b, w in st["segments"]:
            into = st["grad"][w] if w < E else flat[w - E]
            rows = slice(j * nvs + a, j * nvs + b)
            part = d[rows].float().T @ x[rows].float()
            if st["accumulate"]:
                into += part
            else:
                into.copy_(part)
        return dict(grad=st["grad"], slots=st["slots"])
    return _plain_step(st)


def _plain_route(st):
    z, E, K, R, S = st["logits"].float(), st["E"], st["K"], st["R"], st["S"]
    soft, scale, G = st["scoring"] == "softmax", st["scale"], st["groups"]
    n = torch.tensor(st["num_tokens"], device="cuda", dtype=torch.float32)
    valid = torch.arange(S, device="cuda")[None, :, None] < n[:, None, None]

    def score(x):
        if soft:
            return torch.exp(x - x.amax(-1, keepdim=True))
        return 1 / (1 + torch.exp(-x))

    # selection in 64 bits: neighbours in the order may lie a rounding apart
    c = score(z.double())
    if soft:
        c = c / c.sum(-1, keepdim=True)
    if st["bias"] is not None:
        c = c + st["bias"].double()
    if st["top_groups"] < G:
        parts = c.view(R, S, G, E // G)
        if st["group_score"] == "max":
            best = parts.amax(-1)
        else:
            best = torch.sort(parts, dim=-1, descending=True).values[..., :2].sum(-1)
        order = torch.sort(best, dim=-1, descending=True, stable=True).indices
        keep = torch.zeros(R, S, G, dtype=torch.bool, device="cuda")
        keep.scatter_(-1, order[..., :st["top_groups"]], True)
        c = torch.where(keep[..., None], parts, -math.inf).view(R, S, E)
    # a stable order keeps the lowest of equal scores first
    topk = torch.sort(c, dim=-1, descending=True, stable=True).indices[..., :K]
    s = score(z)
    Z = s.sum(-1, keepdim=True)
    p = s / Z
    a = p if soft else s  # what a weight is made of
    ak = a.gather(-1, topk)
    Zk = ak.sum(-1, keepdim=True) if st["renormalize"] else torch.ones_like(ak[..., :1])
    w = torch.where(valid, scale * (ak / Zk), 0.0)
    one = torch.zeros(R, S, E, device="cuda").scatter_(-1, topk, 1.0) * valid
    picks = one.sum(1)
    tpe = picks.to(torch.int32)
    tpe[:, 0] += ((S - n) * K).to(torch.int32)
    out = dict(topk=torch.where(valid, topk, 0).to(torch.int32), weights=w,
               tokens_per_expert=tpe)
    if not st["train"]:
        return out
    prob = (p * valid).sum(1)
    if st["scope"] == "rank":
        groups = (n > 0).sum().clamp(min=1)
        t = n.clamp(min=1)[:, None]
        coef = 1e-4 * E * picks / (K * t * t * groups)
    else:
        t = n.sum().clamp(min=1)
        coef = (1e-4 * E * picks.sum(0) / (K * t * t)).expand(R, E)
    out["loss"] = (coef * prob).sum().reshape(1)
    cf, dw = coef[:, None, :], st["d_weights"]
    if st["renormalize"]:
        # of the picks' raw scores, whose common factor the weights do not see
        sk = s.gather(-1, topk)
        q = sk / sk.sum(-1, keepdim=True)
        dk = scale * (dw - (q * dw).sum(-1, keepdim=True)) / sk.sum(-1, keepdim=True)
        ds = torch.zeros_like(s).scatter_add_(-1, topk, dk)
    else:
        da = torch.zeros_like(s).scatter_add_(-1, topk, scale * dw)
        ds = (da - (p * da).sum(-1, keepdim=True)) / Z if soft else da
    ds = ds + st["d_loss"] * (cf - (p * cf).sum(-1, keepdim=True)) / Z
    dz = ds * s if soft else ds * s * (1 - s)
    out["d_logits"] = torch.where(valid, dz, 0.0).to(st["logits"].dtype)
    if st["biased"]:
        load = picks.sum(0).long()
        st["bias"] += 1e-3 * torch.sign(load.sum() - load * E).float()
        out["bias"] = st["bias"]
    return out


def _pow2(e):
    """2^e in fp32, -149 <= e <= 127, from its bits."""
    bits = torch.where(e > -127, (e + 127) << 23, 1 << (e.clamp(max=-127) + 149))
    return bits.to(torch.int32).view(torch.float32)


def _block_power(v, octaves, most):
    """e of each block of 32: the smallest, at least -127, with |v| <= most 2^(e + octaves)."""
    m, e = torch.frexp(v.view(-1, 32).abs().amax(-1, keepdim=True))
    e = e - 1 - octaves + (m * 2 > most)
    return torch.where(m == 0, torch.full_like(e, -127), e.clamp(min=-127))


def _grid(t, low, r):
    """t >= 0 on the grid of four significant bits and least step 2^(low - 3)."""
    e = (torch.frexp(t)[1] - 1).clamp(min=low) - 3
    q = t * _pow2(-e)
    q = torch.round(q) if r is None else torch.floor(q + r * 2.0 ** -16)
    return q * _pow2(e)


def _encode_m(m, r):
    """E4M3 codes and E8M0 scales."""
    e = _block_power(m, 8, 1.75)
    t = m.view(-1, 32) * _pow2(-e)
    q = torch.copysign(_grid(t.abs(), -6, None if r is None else r.view(-1, 32)), t)
    return q.to(torch.float8_e4m3fn).view(torch.uint8).view(-1), (e + 127).to(torch.uint8).view(-1)


def _encode_v(v, r):
    e = _block_power(v, 30, 1.875)
    t = v.view(-1, 32) * _pow2(-e)
    q = _grid(t, 0, None if r is None else r.view(-1, 32))
    q = torch.where(t > 0, q.clamp(min=0.125), q)
    code = torch.where(q < 1, (q * 8).to(torch.int32),
                       (q.view(torch.int32) >> 20) - (126 << 3))
    return code.to(torch.uint8).view(-1), (e + 127).to(torch.uint8).view(-1)


def _decode(codes, scales, second):
    f = _pow2(scales.int()[:, None] - 127)
    if not second:
        return (codes.view(torch.float8_e4m3fn).float().view(-1, 32) * f).view(-1)
    c = codes.int()
    q = torch.where(c < 8, c.float() / 8, ((c.clamp(min=8) + (126 << 3)) << 20).view(torch.float32))
    return (q.view(-1, 32) * f).view(-1)


_U32 = 0xffffffff


def _mix(x):
    """A 32-bit mixing step on int64 tensors or integers: shifts and odd factors."""
    x = x ^ (x >> 16)
    x = (x * 0x243f6a89) & _U32
    x = x ^ (x >> 15)
    x = (x * 0xb7e15163) & _U32
    return x ^ (x >> 16)


def _words(st):
    """word(seed, step, tensor, element) of every element."""
    key = _mix((_SEED + _mix(_STEP)) & _U32)
    at = torch.arange(st["p"].numel(), device="cuda")
    t = torch.searchsorted(st["first"], at, right=True) - 1
    i = at - st["first"][t]
    key = _mix((key + 0x9e3779b9 * (t + 1)) & _U32)
    return _mix(key ^ (i & _U32) ^ (((i >> 32) * 0x9e3779b9) & _U32))


def _plain_step(st):
    out = {}
    p, g = st["p"].float(), st["g"].float()
    if st["clip"]:
        norm = torch.sqrt((g * g).double().sum()).float().reshape(1)
        out["norm"] = norm
        g = g * (_MAX_NORM / norm).clamp(max=1.0)
    if st["bits"] == 8:
        m8, ms, v8, vs = st["moments"]
        m, v = _decode(m8, ms, False), _decode(v8, vs, True)
    else:
        m, v = st["moments"]
    b1, b2 = _HYPER["betas"]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    lr, wd = _HYPER["lr"], _HYPER["weight_decay"]
    den = torch.sqrt(v) * (1 - b2 ** _STEP) ** -0.5 + _HYPER["eps"]
    p = p * (1 - lr * wd) - (lr / (1 - b1 ** _STEP)) * (m / den)
    r = _words(st) if st["seeded"] else None
    if st["bits"] == 8:
        for to, have in zip(st["moments"], (*_encode_m(m, None if r is None else r & 0xffff),
                                            *_encode_v(v, None if r is None else r >> 16))):
            to.copy_(have)
        out["m"] = _decode(m8, ms, False).bfloat16()
        out["v"] = _decode(v8, vs, True).bfloat16()
    else:
        for to, have in zip(st["moments"], (m, v)):
            to.copy_(have)
        out["m"], out["v"] = st["moments"]
    if st["dtype"] == "bfloat16" and r is not None:
        up = _mix((r + 0x9e3779b9) & _U32) & 0xffff
        p = ((p.view(torch.int32) + up.to(torch.int32)) & -65536).view(torch.float32)
    st["p"].copy_(p)
    out["p"] = st["p"]
    if st["copy"] is not None:
        st["copy"].copy_(p)
        out["copy"] = st["copy"]
    return out


# ----------------------------------------------------------- what it has to do


def work(case):
    c = case
    if c["kind"] == "route":
        tokens = c["R"] * c["S"]
        size = 4 if c["dtype"] == "float32" else 2
        b = tokens * (c["E"] * size + c["K"] * 8) + 4 * c["R"] * c["E"]
        if c["train"]:
            b += tokens * (c["E"] * size + c["K"] * 4)
        return dict(bytes=b, flops=tokens * c["E"] * (16 if c["train"] else 8))
    if c["kind"] == "grad":
        # expected rows with half a padding unit for each home segment; half
        # of the slots are used
        rows = c["R"] * c["C"] + (c["tp"] - 1) * min(c["E"], c["R"] * c["C"]) // 2
        used = c["E"] + c["R"] * c["B"] // 2
        b = rows * (c["N"] + c["Kd"]) * 2 + used * c["N"] * c["Kd"] * (8 if c["accumulate"] else 4)
        return dict(bytes=b, flops=2 * rows * c["N"] * c["Kd"])
    n = sum(_sizes(c)[0])
    size = dict(float32=4, bfloat16=2)
    # the norm has to be known before the first update, so gradients are read
    # twice; moments in 8 bits are read back as the values they stand for
    b = 2 * size[c["dtype"]] + size[c["grad"]] * (2 if c["clip"] else 1) + 2 * c["copy"]
    b += 16 if c["bits"] == 32 else 6 * (1 + 1 / 32) + 4
    return dict(bytes=n * b, flops=n * 20)


# --------------------------------------------------------------- in 64 bits


def exact(case, seed):
    c = dict(case)
    if c["kind"] == "grad" and c["R"] * c["C"] * c["N"] * c["Kd"] > 1 << 41:
        return None  # minutes in 64 bits
    if c["kind"] == "step" and c["elements"] > 1 << 27:
        return None
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if c["kind"] == "route":
        return _exact_route(st)
    if c["kind"] == "grad":
        grad, slots = st["grad"].double(), st["slots"].double()
        both = [grad, slots.view(-1, c["N"], c["Kd"])]
        for j, a, b, w in st["segments"]:
            a, b = j * st["NvS"] + a, j * st["NvS"] + b
            home = w < c["E"]
            both[not home][w if home else w - c["E"]] += torch.einsum(
                "rn,rk->nk", st["d"][a:b].double(), st["x"][a:b].double())
        return dict(grad=grad, slots=slots)
    return _exact_step(st)


def _exact_route(st):
    R, S, E, K, G = st["R"], st["S"], st["E"], st["K"], st["groups"]
    z = st["logits"].double()
    soft = st["scoring"] == "softmax"
    sig = torch.sigmoid(z)
    prob = torch.softmax(z, -1) if soft else sig / sig.sum(-1, keepdim=True)
    kind = prob if soft else sig
    by = kind.cpu().numpy()
    if st["bias"] is not None:
        by = by + st["bias"].double().cpu().numpy()
    if st["top_groups"] < G:
        ranked = -np.sort(-by.reshape(R, S, G, E // G), axis=-1)
        value = ranked[..., 0]
        if st["group_score"] == "top2" and E > G:
            value = value + ranked[..., 1]
        place = np.argsort(np.argsort(-value, axis=-1, kind="stable"), axis=-1, kind="stable")
        out = np.repeat(place >= st["top_groups"], E // G, axis=-1)
        by = np.where(out, -np.inf, by)
    ids = torch.from_numpy(np.argsort(-by, axis=-1, kind="stable")[..., :K].copy()).cuda()
    live = torch.zeros(R, S, dtype=torch.float64, device="cuda")
    for r, n in enumerate(st["num_tokens"]):
        live[r, :n] = 1
    pk = kind.gather(-1, ids)
    share = pk / pk.sum(-1, keepdim=True)
    wt = st["scale"] * (share if st["renormalize"] else pk) * live[..., None]
    out = dict(topk=None, weights=wt, tokens_per_expert=None)
    if not st["train"]:
        return out
    chosen = torch.zeros(R, E, dtype=torch.float64, device="cuda").scatter_add_(
        1, ids.reshape(R, -1), live[..., None].expand(R, S, K).reshape(R, -1))
    mass, n = (prob * live[..., None]).sum(1), live.sum(1)
    coef = torch.zeros(R, E, dtype=torch.float64, device="cuda")
    if st["scope"] == "rank":
        busy = [r for r in range(R) if n[r] > 0]
        for r in busy:
            coef[r] = 1e-4 * (E * chosen[r] / (K * n[r])) / n[r] / len(busy)
    elif n.sum() > 0:
        coef[:] = 1e-4 * (E * chosen.sum(0) / (K * n.sum())) / n.sum()
    out["loss"] = (coef * mass).sum().reshape(1)
    # in the logarithm of the scores, where both scorings have simple slopes
    c = coef[:, None, :] * float(st["d_loss"])
    dlog = prob * (c - (prob * c).sum(-1, keepdim=True))
    dw = st["d_weights"].double()
    term = wt * dw
    if st["renormalize"]:
        term = term - share * term.sum(-1, keepdim=True)
    dlog = dlog + torch.zeros_like(prob).scatter_(-1, ids, term)
    if soft and not st["renormalize"]:
        dlog = dlog - prob * term.sum(-1, keepdim=True)
    slope = 1.0 if soft else torch.sigmoid(-z)  # d log(score) / d logit
    out["d_logits"] = dlog * slope * live[..., None]
    if st["biased"]:
        load = chosen.sum(0)
        # the bias is held in 32 bits and takes its steps there
        out["bias"] = (st["bias"] + 1e-3 * torch.sign(load.mean() - load).float()).double()
    return out


def _exact_on(values, x, up):
    """|x| on the ascending `values`: the nearest, ties to the even place, or
    with `up` in [0, 1) by where x lies between its neighbours."""
    hi = torch.searchsorted(values, x).clamp(1, len(values) - 1)
    a, b = values[hi - 1], values[hi]
    part = (x - a) / (b - a)
    if up is None:
        take = (part > 0.5) | ((part == 0.5) & (hi % 2 == 0))
    else:
        take = part + up >= 1
    return torch.where(take, b, a)


def _exact_step(st):
    c = st
    g, p = st["g"].double(), st["p"].double()
    norm = torch.linalg.vector_norm(g)
    out = {}
    if c["clip"]:
        out["norm"] = norm.reshape(1)
        g = g * min(1.0, _MAX_NORM / float(norm))
    two = torch.tensor([2.0 ** (b - 127) for b in range(256)], dtype=torch.float64, device="cuda")
    e4m3 = torch.tensor([n % 8 * 2.0 ** -9 if n < 8 else (8 + n % 8) * 2.0 ** (n // 8 - 10)
                         for n in range(127)], dtype=torch.float64, device="cuda")
    e5m3 = torch.tensor([n / 8 if n < 8 else (8 + n % 8) * 2.0 ** (n // 8 - 4)
                         for n in range(256)], dtype=torch.float64, device="cuda")
    if c["bits"] == 8:
        m8, ms, v8, vs = st["moments"]
        b = m8.long()
        m = e4m3[b & 127] * torch.where(b > 127, -1.0, 1.0)
        m = (m.view(-1, 32) * two[ms.long()][:, None]).view(-1)
        v = (e5m3[v8.long()].view(-1, 32) * two[vs.long()][:, None]).view(-1)
    else:
        m, v = (t.double() for t in st["moments"])
    b1, b2 = _HYPER["betas"]
    m, v = m + (1 - b1) * (g - m), v + (1 - b2) * (g ** 2 - v)
    p = p - _HYPER["lr"] * (_HYPER["weight_decay"] * p + (m / (1 - b1 ** _STEP)) / (
        torch.sqrt(v / (1 - b2 ** _STEP)) + _HYPER["eps"]))
    word = None
    if c["seeded"]:
        word = np.zeros(p.numel(), np.uint32)
        golden = np.uint32(0x9e3779b9)

        def stir(x):
            x = x ^ (x >> np.uint32(16))
            x = x * np.uint32(0x243f6a89)
            x = x ^ (x >> np.uint32(15))
            x = x * np.uint32(0xb7e15163)
            return x ^ (x >> np.uint32(16))

        with np.errstate(over="ignore"):
            start = stir(np.array([_SEED], np.uint32) + stir(np.array([_STEP], np.uint32)))
            sizes, first = _sizes(c)
            for k, (a, s) in enumerate(zip(first, sizes)):
                key = stir(start + golden * np.uint32(k + 1))
                word[a:a + s] = stir(key ^ np.arange(s, dtype=np.uint32))
            more = stir(word + golden)
        up = lambda x: torch.from_numpy(x.astype(np.float64) / 65536).cuda()  # noqa: E731
    if c["bits"] == 8:
        out["m"], out["v"] = (
            _exact_moment(x, values, two, None if word is None else up(bits))
            for x, values, bits in ((m, e4m3, word & 0xffff if word is not None else None),
                                    (v, e5m3, word >> 16 if word is not None else None)))
    else:
        out["m"], out["v"] = m, v
    if c["dtype"] == "bfloat16" and word is not None:
        _, e = torch.frexp(p)
        unit = 2.0 ** (e.double() - 8)
        p = torch.copysign(torch.floor(p.abs() / unit + up(more & 0xffff)) * unit, p)
    out["p"] = p
    if c["copy"] is not None:
        out["copy"] = p
    return out


def _exact_moment(x, values, two, up):
    """The 8-bit moments' values: each block of 32 under the smallest power of
    two that holds it."""
    x = x.view(-1, 32)
    top = x.abs().amax(1)
    unit = two[torch.searchsorted(two * values[-1], top).clamp(max=254)][:, None]
    a = x.abs() / unit
    q = _exact_on(values, a, None if up is None else up.view(-1, 32))
    if len(values) == 256:  # the second moment stays above zero
        q = torch.where(a > 0, q.clamp(min=float(values[1])), q)
    return (torch.copysign(q, x) * unit).view(-1)
