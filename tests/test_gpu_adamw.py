"""AdamW over many tensors, its 8-bit moments and the gradients' norm on the
GPU, against their 64-bit forms.

fp32 arithmetic rounds each operation by 2^-24 at most.  m and v take three
operations on their terms (2^-24 each, on values no larger than the terms'
magnitudes' sum), so |error| <= 4 2^-24 (b1 |m| + (1 - b1) |g|); the update's
quotient adds the square root's and the inverse's approximations (2^-22 each),
a product, a sum and m's and v's own errors: 2^-19 of the update is an upper
bound, and p adds its two roundings, 2^-23 |p|.  Hyperparameters rounded to fp32
add 2^-24 relative each and are inside those bounds, except 1 - b2: it is
computed in 64 bits, so it is one rounding too.
"""
import numpy as np
import pytest
import torch

from tests import train_refs as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HYPER = dict(lr=3e-3, betas=(0.9, 0.99), eps=1e-7, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.fixture(scope="module")
def buf():
    from combine_moonep_plan_gb300 import Buffer
    return Buffer(S=1, H=8, K=1, E=1, num_ep_ranks=1, zero_copy_views=False)


def _f64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def _tensors(sizes, dtype, seed, std, shift):
    """Tensors of `sizes`; with shift they start one element off a vector."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for n in sizes:
        t = torch.randn(n + shift, generator=g, device="cuda") * std
        out.append(t.to(dtype)[shift:])
    return out


def _check_p(got, want, old, lr, dtype, extra=0.0):
    upd = np.abs(want - old * (1 - HYPER["lr"] * HYPER["weight_decay"]))
    tol = 2.0 ** -19 * upd + 4 * U * np.abs(old) + extra
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want) + 1e-40
    assert np.all(np.abs(got - want) <= tol)


SIZES = [1, 7, 8, 31, 32, 33, 0, 2047, 2048, 2049, 12345]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("clip", [False, True])
def test_steps_32_bits(buf, dtype, gtype, shift, clip):
    params = _tensors(SIZES, dtype, 1, 0.5, shift)
    weights = [torch.zeros(n + shift, device="cuda").bfloat16()[shift:] for n in SIZES]
    if dtype == torch.bfloat16:
        weights = None
    else:
        weights[3] = None
    state = buf.adamw_state(params)
    for step in range(1, 4):
        grads = _tensors(SIZES, gtype, 10 + step, 2.0, shift)
        old = [_f64(t) for t in params]
        mom = [(_f64(a), _f64(b)) for a, b in zip(*(state.split(t) for t in state.tensors))]
        kw, norm, most = {}, None, None
        if clip:
            most = 1.5
            kw = dict(norm=buf.grad_norm(grads), max_norm=most)
            norm = kw["norm"].item()
            full = np.sqrt(sum((_f64(t) ** 2).sum() for t in grads))
            # sums of eight in fp32, each square rounded: 9 roundings, halved by the root
            assert abs(norm - full) <= 6 * U * full
        buf.adamw(params, grads, state, step=step, weights=weights, **HYPER, **kw)
        for k, n in enumerate(SIZES):
            g = _f64(grads[k])
            p, m, v = ref.adamw(old[k], g, *mom[k], step, HYPER["lr"], *HYPER["betas"],
                                HYPER["eps"], HYPER["weight_decay"], norm, most)
            s = min(1, most / norm) if clip else 1.0
            b1, b2 = HYPER["betas"]
            gm, gv = state.split(state.tensors[0])[k], state.split(state.tensors[1])[k]
            # with a clip the factor has two roundings more, squared in v
            assert np.all(np.abs(_f64(gm) - m) <= 6 * U * (
                b1 * np.abs(mom[k][0]) + (1 - b1) * s * np.abs(g)))
            assert np.all(np.abs(_f64(gv) - v) <= 10 * U * v)
            # m's own error relative to its terms can exceed 2^-19 of the update
            # where they cancel
            err = HYPER["lr"] / (1 - b1 ** step) * 6 * U * (
                b1 * np.abs(mom[k][0]) + (1 - b1) * s * np.abs(g)) / (
                np.sqrt(v / (1 - b2 ** step)) + HYPER["eps"])
            _check_p(_f64(params[k]), p, old[k], HYPER["lr"], dtype, 2 * err)
            if weights is not None and weights[k] is not None:
                assert torch.equal(weights[k], params[k].bfloat16())
    assert buf.get_status() == 0
    # what pads a tensor's moments to whole blocks stays zero
    for t in state.tensors:
        for o, n in zip(state.offsets, state.sizes):
            assert not t[o + n:o + -(-n // 32) * 32].any()


@pytest.mark.parametrize("seed", [None, 5])
@pytest.mark.parametrize("dtype,gtype,shift", [(torch.float32, torch.float32, 0),
                                               (torch.float32, torch.bfloat16, 1),
                                               (torch.bfloat16, torch.float32, 1),
                                               (torch.bfloat16, torch.bfloat16, 0)])
def test_steps_8_bits(buf, seed, dtype, gtype, shift):
    """The new moments, from the old ones' values in 64 bits, are off by at
    most half a step of the grid (a whole one when rounded at random)."""
    params = _tensors(SIZES, dtype, 2, 0.5, shift)
    state = buf.adamw_state(params, bits=8)
    b1, b2 = HYPER["betas"]
    for step in range(1, 5):
        grads = _tensors(SIZES, gtype, 20 + step, 10.0 ** (3 - 2 * step), shift)
        if step == 3:
            grads[9].zero_()
        old = [_f64(t) for t in params]
        codes = [t.cpu().numpy() for t in state.tensors]
        m0, v0 = (ref.moment_decode(codes[2 * i], codes[2 * i + 1], i) for i in (0, 1))
        buf.adamw(params, grads, state, step=step, seed=seed, **HYPER)
        codes = [t.cpu().numpy() for t in state.tensors]
        m1, v1 = (ref.moment_decode(codes[2 * i], codes[2 * i + 1], i) for i in (0, 1))
        flat_m, flat_v = state.moments(torch.float32)
        assert np.array_equal(_f64(flat_m), m1)
        # the least codes' values are subnormal in fp32 only below 2^-126
        assert np.array_equal(_f64(flat_v), v1)
        g = np.zeros(state.total)
        for o, n, t in zip(state.offsets, SIZES, grads):
            g[o:o + n] = _f64(t)
        m, v = b1 * m0 + (1 - b1) * g, b2 * v0 + (1 - b2) * g * g
        for x, got, second, scales in ((m, m1, 0, codes[1]), (v, v1, 1, codes[3])):
            want = ref.moment_scale(x, second)
            edge = ref.moment_scale(x * (1 + 2.0 ** -20), second)
            edge2 = ref.moment_scale(x * (1 - 2.0 ** -20), second)
            assert np.all((scales == want) | (scales == edge) | (scales == edge2))
            unit = ref.moment_step(x, scales, second)
            slack = 8 * U * (b1 * np.abs(m0) + np.abs(g)) if not second else 16 * U * v
            off = np.abs(got - x)
            assert np.all(off <= unit * (0.5 if seed is None else 1.0) + slack
                          + (unit if second else 0) * (x > 0) * (got == unit))
            if second:
                assert np.all((got > 0) == (x > 0))
        for k, (o, n) in enumerate(zip(state.offsets, SIZES)):
            p, _, _ = ref.adamw(old[k], g[o:o + n], m0[o:o + n], v0[o:o + n], step, HYPER["lr"],
                                b1, b2, HYPER["eps"], HYPER["weight_decay"])
            den = np.sqrt(v[o:o + n] / (1 - b2 ** step)) + HYPER["eps"]
            err = HYPER["lr"] / (1 - b1 ** step) * 6 * U * (
                b1 * np.abs(m0[o:o + n]) + (1 - b1) * np.abs(g[o:o + n])) / den
            if dtype == torch.bfloat16 and seed is not None:
                err = err + 2.0 ** -7 * np.abs(p)  # a whole step
            _check_p(_f64(params[k]), p, old[k], HYPER["lr"], dtype, 2 * err)
    assert buf.get_status() == 0


def test_random_rounding_is_right_on_average(buf):
    """Over 4096 seeds the mean of a rounded value lies within six standard
    errors of it: at most half a step each, so 6 * 0.5 / 64 of a step."""
    n, seeds = 64, 4096
    g = torch.linspace(0.3, 1.7, n, device="cuda")
    want_m, want_v = 0.1 * _f64(g), 0.01 * _f64(g) ** 2
    one = torch.ones(n, device="cuda")
    sums = [np.zeros(n) for _ in range(3)]
    for seed in range(seeds):
        p = one.bfloat16()
        state = buf.adamw_state([p], bits=8)
        buf.adamw([p], [g], state, step=1, seed=seed, **HYPER)
        for s, t in zip(sums, (*state.moments(torch.float32), p)):
            s += _f64(t)
    codes = [t.cpu().numpy() for t in state.tensors]
    for mean, want, second in ((sums[0] / seeds, want_m, 0), (sums[1] / seeds, want_v, 1)):
        unit = ref.moment_step(want, codes[1 + 2 * second], second)
        assert np.all(np.abs(mean - want) <= 6 * 0.5 / 64 * unit)
    want_p, _, _ = ref.adamw(np.ones(n), _f64(g), np.zeros(n), np.zeros(n), 1, HYPER["lr"],
                             *HYPER["betas"], HYPER["eps"], HYPER["weight_decay"])
    assert np.all(np.abs(sums[2] / seeds - want_p) <= 6 * 0.5 / 64 * 2.0 ** -8)
    # other elements, tensors, steps and seeds draw other words
    p = [torch.zeros(4096, device="cuda").bfloat16() for _ in range(2)]
    g = [torch.full((4096,), 1.01, device="cuda") for _ in range(2)]
    got = []
    for seed, step in ((1, 1), (1, 2), (2, 1)):
        state = buf.adamw_state(p, bits=8)
        buf.adamw([t.clone() for t in p], g, state, lr=0.0, step=step, seed=seed, betas=(0.9, 0.9),
                  weight_decay=0.0)
        m = state.split(state.tensors[0])
        got += [m[0], m[1]]
    for i in range(6):
        share = (got[i] != got[i][0]).float().mean().item()
        assert 0.05 < share < 0.95
        for j in range(i):
            assert not torch.equal(got[i], got[j])


def test_second_moment_follows_small_changes(buf):
    """At beta2 = 0.999 a step moves v by 0.1 %, a hundredth of its grid: random
    rounding lets it decay (0.999^700 = 0.496), rounding to nearest holds it."""
    n = 4096
    p, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    v = {}
    for seed in (None, 3):
        state = buf.adamw_state([p], bits=8)
        buf.adamw([p.clone()], [g], state, lr=0.0, step=1, seed=seed)
        v0 = state.moments(torch.float32)[1].mean().item()
        for step in range(2, 702):
            buf.adamw([p], [torch.zeros_like(g)], state, lr=0.0, step=step, seed=seed)
        v[seed] = state.moments(torch.float32)[1].mean().item() / v0
    assert v[None] > 0.99
    # each value's spread is at most its own size: 1/64 of it for the mean, 6 of those
    assert abs(v[3] - 0.999 ** 700) <= 6 / 64


def test_many_tensors(buf):
    """More tensors than one launch takes, some empty, unaligned ones between."""
    sizes = [(37 * i) % 71 for i in range(801)]
    params = _tensors(sizes, torch.float32, 3, 1.0, 0)
    grads = _tensors(sizes, torch.float32, 4, 1.0, 0)
    grads[5] = torch.randn(sizes[5] + 1, device="cuda")[1:]
    one = [torch.cat([t.reshape(-1) for t in x]) for x in (params, grads)]
    a, b = buf.adamw_state(params), buf.adamw_state([one[0]])
    norm = buf.grad_norm(grads)
    full = np.sqrt((_f64(one[1]) ** 2).sum())
    assert abs(norm.item() - full) <= 6 * U * full
    for step in (1, 2):
        buf.adamw(params, grads, a, step=step, norm=norm, max_norm=1.0, **HYPER)
        buf.adamw([one[0]], [one[1]], b, step=step, norm=norm, max_norm=1.0, **HYPER)
    assert torch.equal(torch.cat([t.reshape(-1) for t in params]), one[0])
    for x, y in zip(a.tensors, b.tensors):
        assert torch.equal(torch.cat(a.split(x)), b.split(y)[0])
    assert buf.grad_norm([]).item() == 0 and buf.grad_norm([one[0][:0]]).item() == 0
    buf.adamw([], [], buf.adamw_state([]), lr=1.0, step=1)
    assert torch.equal(buf.grad_norm(grads), norm)  # a fixed order


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_norm_changes_nothing(buf, bad):
    p, g = torch.randn(1000, device="cuda"), torch.randn(1000, device="cuda")
    w = torch.zeros(1000, device="cuda").bfloat16()
    for bits in (32, 8):
        state = buf.adamw_state([p], bits=bits)
        buf.adamw([p], [g], state, step=1, weights=[w], **HYPER)
        g2 = g.clone()
        g2[17] = bad
        norm = buf.grad_norm([g2])
        assert not norm.isfinite().item()
        before = [t.clone() for t in (p, w, *state.tensors)]
        buf.adamw([p], [g2], state, step=2, norm=norm, max_norm=1.0, weights=[w], **HYPER)
        for x, y in zip(before, (p, w, *state.tensors)):
            assert torch.equal(x, y)
    # without a norm it goes where the formula takes it; 8 bits: its whole block
    state = buf.adamw_state([p], bits=8)
    buf.adamw([p], [g2], state, step=1, seed=1, **HYPER)
    m, v = state.moments(torch.float32)
    assert m[0:32].isnan().all() and v[0:32].isnan().all()
    assert m[32:].isfinite().all() and v[32:].isfinite().all()
    assert p[:17].isfinite().all() and p[18:].isfinite().all()


def test_captured_step_with_device_scalars(buf):
    """A captured step reads its number and rate anew: as eager steps."""
    p = [torch.randn(n, device="cuda") for n in (1000, 77)]
    g = [torch.randn(n, device="cuda") for n in (1000, 77)]
    q = [t.clone() for t in p]
    a, b = buf.adamw_state(p, bits=8), buf.adamw_state(q, bits=8)
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    lr = torch.zeros(1, device="cuda")
    kw = dict(betas=(0.9, 0.95), weight_decay=0.1, seed=9)

    def one():
        step.add_(1)
        norm = buf.grad_norm(g)
        buf.adamw(p, g, a, lr=lr, step=step, norm=norm, max_norm=2.0, **kw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        one()
    for k in range(1, 6):
        lr.fill_(1e-2 / k)
        for t in g:
            t.normal_()
        graph.replay()
        norm = buf.grad_norm(g)
        buf.adamw(q, g, b, lr=1e-2 / k, step=k, norm=norm, max_norm=2.0, **kw)
        for x, y in zip(a.tensors, b.tensors):
            assert torch.equal(x, y)
        for x, y in zip(p, q):
            # rate and root: a few fp32 roundings each, of an update below 5 lr
            assert (x - y).abs().max().item() <= 2.0 ** -18 * 5e-2
    assert step.item() == 5 and buf.get_status() == 0


def test_few_sms(buf):
    """A context of one SM takes the same steps."""
    from combine_moonep_plan_gb300 import Buffer
    one = Buffer(S=1, H=8, K=1, E=1, num_ep_ranks=1, zero_copy_views=False, num_sms=1)
    for bits, dtype in ((32, torch.float32), (8, torch.float32), (8, torch.bfloat16)):
        p = _tensors([100000, 33, 4097], dtype, 1, 1.0, 0)
        g = _tensors([100000, 33, 4097], torch.float32, 2, 1.0, 0)
        got = []
        for b in (buf, one):
            q = [t.clone() for t in p]
            state = b.adamw_state(q, bits=bits)
            norm = b.grad_norm(g)
            b.adamw(q, g, state, step=1, seed=3, norm=norm, max_norm=1.0, **HYPER)
            got.append((*q, *state.tensors, *state.moments()))
            full = np.sqrt(sum((_f64(t) ** 2).sum() for t in g))
            assert abs(norm.item() - full) <= 6 * U * full
        # the norm's sums are split over the blocks, so its last bit may differ, which
        # may move a clipped value by one, and a rounded one by a step in a million
        for x, y in zip(*got):
            assert (x != y).float().mean().item() <= (1.0 if x.dtype == torch.float32 else 1e-3)
            if x.dtype == torch.float32:
                assert torch.allclose(x, y, rtol=2.0 ** -20, atol=2.0 ** -20)


def test_device_step_below_one_counts_as_one(buf):
    p, g = torch.ones(100, device="cuda"), torch.randn(100, device="cuda")
    q = p.clone()
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = buf.adamw_state([p]), buf.adamw_state([q])
    buf.adamw([p], [g], a, lr=0.1, step=zero)
    buf.adamw([q], [g], b, lr=0.1, step=1)
    assert torch.allclose(p, q, rtol=2.0 ** -20) and torch.equal(a.tensors[0], b.tensors[0])


def test_past_two_to_31_elements(buf):
    n = (1 << 31) + 1000
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[-5:] = 1.0
    g[-5:] = 0.5
    g[3] = 2.0
    state = buf.adamw_state([p], bits=8)
    norm = buf.grad_norm([g])
    assert abs(norm.item() - np.sqrt(4 + 5 * 0.25)) <= 6 * U * 3
    buf.adamw([p], [g], state, lr=0.125, step=1, weight_decay=0.0, seed=1)
    # the first step is lr * sign(g); random rounding leaves these whole values or moves
    # them by one bf16 step, 2^-8
    assert (p[-5:].float() - 0.875).abs().max().item() <= 2.0 ** -8
    assert abs(p[3].item() + 0.125) <= 2.0 ** -10
    assert p.count_nonzero().item() == 6
    m8, _, v8, _ = state.tensors
    assert m8.count_nonzero().item() == 6 and v8.count_nonzero().item() == 6


def test_refusals(buf):
    p, g = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    s = buf.adamw_state([p])
    from combine_moonep_plan_gb300._lib import MoonepError
    with pytest.raises(ValueError):
        buf.adamw_state([p], bits=16)
    with pytest.raises(TypeError):
        buf.adamw_state([p.half()])
    with pytest.raises(TypeError):
        buf.adamw([p, p.bfloat16()], [g, g], buf.adamw_state([p, p]), lr=1, step=1)
    with pytest.raises(ValueError):
        buf.adamw([p, p], [g, g], buf.adamw_state([p, p]), lr=1, step=1)
    with pytest.raises(ValueError):
        buf.adamw([p], [g, g], s, lr=1, step=1)
    with pytest.raises(ValueError):
        buf.adamw([p], [g[:63]], s, lr=1, step=1)
    with pytest.raises(ValueError):
        buf.adamw([p], [torch.zeros(128, device="cuda")[::2]], s, lr=1, step=1)
    with pytest.raises(ValueError):
        buf.adamw([p.cpu()], [g], s, lr=1, step=1)
    with pytest.raises(ValueError):
        buf.adamw([p], [g], s, lr=1, step=0)
    with pytest.raises(ValueError):
        buf.adamw([p], [g], s, lr=1, step=1, max_norm=1.0)
    with pytest.raises(TypeError):
        buf.adamw([p], [g], s, lr=1, step=torch.ones(1, device="cuda"))
    with pytest.raises(TypeError):
        buf.adamw([p.bfloat16()], [g], s, lr=1, step=1, weights=[p.bfloat16()])
    nan = float("nan")
    for kw in (dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=0.0), dict(eps=1e-60),
               dict(betas=(nan, 0.9)), dict(weight_decay=nan)):
        with pytest.raises(MoonepError):
            buf.adamw([p], [g], s, **{**dict(lr=1, step=1), **kw})
    for lr, most in ((nan, 1.0), (float("inf"), 1.0), (1.0, 0.0), (1.0, nan)):
        with pytest.raises(MoonepError):
            buf.adamw([p], [g], s, lr=lr, step=1, norm=buf.grad_norm([g]), max_norm=most)
    assert not p.any() and not s.tensors[0].any()
