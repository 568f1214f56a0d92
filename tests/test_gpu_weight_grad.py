"""The experts' weight gradients on the GPU against their 64-bit form.

Products of bf16 values are exact in fp32.  The tensor cores add 16 rows at a
time to the fp32 sum; with each addition off by at most 2^-22 of the terms'
magnitudes' sum (alignment of the terms and the sum to a common exponent,
without rounding to nearest), a sum over n rows is off by (n / 16 + 2) 2^-22 of
it, and an addition to an earlier gradient by 2^-24 of the result more.
"""
import numpy as np
import pytest
import torch

from tests import train_refs as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _buffer(R, E, B, S, **kw):
    from combine_moonep_plan_gb300 import Buffer
    return Buffer(S=S, H=8, K=1, E=E, num_ep_ranks=R, B=B, token_padding=1,
                  zero_copy_views=False, **kw)


def _cu(R, E, B, lengths, NvS):
    """cu_seqlens of segments of these lengths, taken in turn by the segments
    that a rank may hold."""
    cu = np.zeros((R, E + B), np.int32)
    L, at = E // R, 0
    for j in range(R):
        size = np.zeros(E + B, np.int64)
        for x in [*range(j * L, (j + 1) * L), *range(E, E + B)]:
            size[x] = lengths[at % len(lengths)]
            at += 1
        cu[j] = np.cumsum(size)
    assert cu.max() <= NvS
    return cu


def _check(buf, cu, N, Kd, seed=0, accumulate=False, pad=0, garbage=True):
    R, E, B, NvS = buf.R, buf.E, buf.B, buf.NvS
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = R * NvS
    x = torch.randn(n, Kd + pad, generator=g, device="cuda").bfloat16()
    d = torch.randn(n, N + pad, generator=g, device="cuda").bfloat16()
    if garbage:
        used = torch.zeros(n, dtype=torch.bool, device="cuda")
        for j in range(R):
            used[j * NvS:j * NvS + int(cu[j, -1])] = True
        x[~used], d[~used] = float("nan"), float("inf")
    x, d = x[:, :Kd], d[:, :N]
    grad = torch.full((E, N, Kd), 3.0, device="cuda")
    slots = torch.full((R, B, N, Kd), 5.0, device="cuda")
    if accumulate:
        grad.normal_(generator=g)
        slots.normal_(generator=g)
    old = [t.double().cpu().numpy().reshape(-1, N, Kd) for t in (grad, slots)]
    out = buf.expert_weight_grad(x, d, torch.from_numpy(cu).cuda(), out=(grad, slots),
                                 accumulate=accumulate)
    assert out[0] is grad and out[1] is slots
    got = [t.double().cpu().numpy().reshape(-1, N, Kd) for t in out]
    xn, dn = x.float().cpu().numpy(), d.float().cpu().numpy()
    want, mag = ref.weight_grad(xn, dn, cu, E, R, B, NvS)
    rows = {g: m for g, _, m in ref.ref.segments(cu, E, R, B, NvS)}
    for w in range(E + R * B):
        home = w < E
        have = got[not home][w if home else w - E]
        base = old[not home][w if home else w - E]
        if w not in want:
            assert np.array_equal(have, base if accumulate or not home else 0 * base)
            continue
        total = want[w] + (base if accumulate else 0)
        tol = (rows[w] / 16 + 2) * 2.0 ** -22 * mag[w] + 2.0 ** -24 * np.abs(total)
        assert np.all(np.abs(have - total) <= tol), (w, rows[w], np.abs(have - total).max())
    assert buf.get_status() == 0


LENGTHS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 320, 333]


@pytest.mark.parametrize("N,Kd", [(8, 8), (256, 256), (264, 72), (512, 1000), (1000, 520),
                                  (64, 64), (192, 8), (320, 448)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_lengths(N, Kd, accumulate):
    buf = _buffer(2, 8, 3, 2000)
    for turn in range(3):
        lengths = LENGTHS[turn * 5:] + LENGTHS[:turn * 5]
        _check(buf, _cu(2, 8, 3, lengths, buf.NvS), N, Kd, seed=turn, accumulate=accumulate)


@pytest.mark.parametrize("R,E,B,lengths", [
    (1, 1, 0, [0]), (1, 1, 0, [1]), (1, 1, 1, [700, 5]), (4, 4, 0, [16]), (3, 21, 4, [7, 0, 0, 33]),
    (8, 8, 1, [0]), (1, 3, 2, [0, 90, 0, 40, 0])])
def test_layouts(R, E, B, lengths):
    buf = _buffer(R, E, B, 800)
    cu = _cu(R, E, B, lengths, buf.NvS)
    _check(buf, cu, 272, 144, seed=E)
    _check(buf, cu, 272, 144, seed=E, accumulate=True, pad=8)


def test_more_groups_than_table_entries():
    buf = _buffer(4, 1500, 7, 900)
    _check(buf, _cu(4, 1500, 7, [2, 0, 3, 0, 1], buf.NvS), 16, 40)
    buf = _buffer(2, 4096, 3, 500)
    _check(buf, _cu(2, 4096, 3, [0] * 9 + [2], buf.NvS), 8, 16, accumulate=True)


@pytest.mark.parametrize("sms", [1, 2, 7])
def test_few_sms(sms):
    """One pair of SMs or a few walk all tiles: many per pair, several batches."""
    buf = _buffer(2, 8, 3, 1000, num_sms=sms)
    cu = _cu(2, 8, 3, [64, 17, 0, 33, 128, 80], buf.NvS)
    _check(buf, cu, 1024, 1032, seed=sms)


@pytest.mark.parametrize("N,Kd", [(2056, 264), (4360, 8), (2304, 520)])
def test_more_tiles_than_a_band(N, Kd):
    buf = _buffer(1, 3, 0, 200)
    _check(buf, _cu(1, 3, 0, [70, 0, 33], buf.NvS), N, Kd)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("N,Kd", [(264, 72), (8, 8), (256, 512)])
def test_shares_of_long_segments(N, Kd, accumulate):
    """Few small gradients over many rows: each is computed in shares of its rows."""
    from combine_moonep_plan_gb300 import _lib
    buf = _buffer(2, 4, 1, 6000)
    n = _lib.load().moonep_expert_weight_grad_workspace(buf._ctx, N, Kd)
    assert n >= 2 * 6 * N * Kd * 4 and n % (6 * N * Kd * 4) == 0
    for turn, lengths in enumerate(([2500, 0, 1, 700, 63, 512], [5900, 3, 0, 65, 17, 3001],
                                    [0], [64, 320, 1900])):
        _check(buf, _cu(2, 4, 1, lengths, buf.NvS), N, Kd, seed=turn, accumulate=accumulate)
    # the same twice, and from a capture
    cu = torch.from_numpy(_cu(2, 4, 1, [2500, 0, 1, 700, 63, 512], buf.NvS)).cuda()
    x, d = (torch.randn(2 * buf.NvS, c, device="cuda").bfloat16() for c in (Kd, N))
    first = buf.expert_weight_grad(x, d, cu)
    out = tuple(torch.zeros_like(t) for t in first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        buf.expert_weight_grad(x, d, cu, out=out)
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_long_segment():
    """Twenty thousand rows into one gradient."""
    buf = _buffer(1, 2, 0, 20011)
    _check(buf, np.array([[20000, 20011]], np.int32), 128, 256)


def test_repeats_bit_for_bit_and_overlaps_itself():
    buf = _buffer(2, 8, 2, 1500)
    cu = torch.from_numpy(_cu(2, 8, 2, [300, 77, 0, 150], buf.NvS)).cuda()
    n = 2 * buf.NvS
    x, d = (torch.randn(n, c, device="cuda").bfloat16() for c in (512, 768))
    first = [t.clone() for t in buf.expert_weight_grad(x, d, cu)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            outs += [buf.expert_weight_grad(x, d, cu) for _ in range(3)]
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out[0], first[0]) and torch.equal(out[1], first[1])
    # captured and replayed on new inputs
    graph = torch.cuda.CUDAGraph()
    out = tuple(torch.zeros_like(t) for t in first)
    with torch.cuda.graph(graph):
        buf.expert_weight_grad(x, d, cu, out=out, accumulate=True)
    graph.replay()
    assert torch.equal(out[0], first[0]) and torch.equal(out[1], first[1])
    graph.replay()
    assert torch.equal(out[0], 2 * first[0])
    x.mul_(2)
    graph.replay()
    assert torch.equal(out[0], 4 * first[0])
    assert buf.get_status() == 0


def test_no_rows_at_all():
    """A context without tokens: zeros for the home experts, or nothing added."""
    buf = _buffer(1, 3, 0, 0)
    assert buf.NvS == 0
    x, d = (torch.zeros(0, c, device="cuda").bfloat16() for c in (16, 8))
    cu = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    grad, slots = torch.ones(3, 8, 16, device="cuda"), torch.ones(1, 0, 8, 16, device="cuda")
    buf.expert_weight_grad(x, d, cu, out=(grad, slots), accumulate=True)
    assert grad.eq(1).all()
    buf.expert_weight_grad(x, d, cu, out=(grad, slots))
    assert not grad.any()


def test_beside_a_product_on_another_stream():
    """Two kernels that each want whole SMs take turns."""
    buf = _buffer(2, 8, 2, 3000)
    cu = torch.from_numpy(_cu(2, 8, 2, [500, 77, 0, 450], buf.NvS)).cuda()
    n = 2 * buf.NvS
    x, d = (torch.randn(n, c, device="cuda").bfloat16() for c in (512, 768))
    x4 = buf.quantize_mx(x)
    w4 = buf.quantize_mx(torch.randn(8 + 4, 768, 512, device="cuda").bfloat16())
    grad, _ = buf.expert_weight_grad(x, d, cu)
    y = torch.zeros(n, 768, device="cuda")
    buf.expert_product(x4, w4, cu, out=y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        y2 = torch.zeros_like(y)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            buf.expert_product(x4, w4, cu, out=y2)
        again, _ = buf.expert_weight_grad(x, d, cu)
        torch.cuda.synchronize()
        assert torch.equal(again, grad) and torch.equal(y2, y)
    assert buf.get_status() == 0


def test_against_differences():
    """sum(c * (x W^T)) moves by h times the gradient, with c as d_out: linear, so
    the difference is exact but for 64-bit rounding; the kernel's part is that of
    the 64-bit form above."""
    buf = _buffer(1, 2, 0, 40)
    cu = np.array([[19, 40]], np.int32)
    x = torch.randn(buf.NvS, 16, device="cuda").bfloat16()
    c = torch.randn(buf.NvS, 8, device="cuda").bfloat16()
    grad, _ = buf.expert_weight_grad(x, c, torch.from_numpy(cu).cuda())
    xn, cn = (t.double().cpu().numpy() for t in (x, c))
    W = np.random.default_rng(0).standard_normal((2, 8, 16))

    def value(W):
        return sum((cn[rows] * (xn[rows] @ W[e].T)).sum()
                   for e, rows in enumerate((slice(0, 19), slice(19, 40))))

    for i in np.ndindex(2, 8, 16):
        up = W.copy()
        up[i] += 1.0
        diff = value(up) - value(W)
        rows = slice(0, 19) if i[0] == 0 else slice(19, 40)
        mag = np.abs(cn[rows, i[1]] * xn[rows, i[2]]).sum()
        assert abs(grad[i].item() - diff) <= 4 * 2.0 ** -22 * mag + 1e-10


def test_reported_segments_count_as_empty():
    from combine_moonep_plan_gb300._lib import ERR_PLAN
    buf = _buffer(1, 4, 0, 100)
    x, d = (torch.ones(buf.NvS, c, device="cuda").bfloat16() for c in (16, 8))
    cu = torch.tensor([[10, 5, 30, 1 << 20]], dtype=torch.int32, device="cuda")
    grad, _ = buf.expert_weight_grad(x, d, cu)
    assert grad[0].eq(10).all() and not grad[1].any() and grad[2].eq(25).all() and not grad[3].any()
    assert buf.get_status() == ERR_PLAN and buf.get_status() == 0


def test_past_two_to_31_values():
    """Rows and gradients past 2^31 values."""
    buf = _buffer(1, 3, 0, 1100000)
    n, N, Kd = buf.NvS, 8, 2048
    x = torch.zeros(n, Kd, dtype=torch.bfloat16, device="cuda")
    d = torch.zeros(n, N, dtype=torch.bfloat16, device="cuda")
    x[-3:], d[-3:] = 0.5, 2.0
    cu = torch.tensor([[5, n - 3, n]], dtype=torch.int32, device="cuda")
    grad, _ = buf.expert_weight_grad(x, d, cu)
    assert not grad[:2].any() and grad[2].eq(3.0).all()
    del x, d, grad
    buf = _buffer(1, 5, 0, 100)
    N, Kd = 20480, 32768
    x = torch.randn(buf.NvS, Kd, device="cuda").bfloat16()
    d = torch.randn(buf.NvS, N, device="cuda").bfloat16()
    cu = torch.tensor([[20, 40, 60, 80, 100]], dtype=torch.int32, device="cuda")
    grad, _ = buf.expert_weight_grad(x, d, cu)
    for e in (0, 4):
        a = slice(20 * e, 20 * e + 20)
        for n0, k0 in ((0, 0), (N - 8, Kd - 8), (12000, 5000)):
            want = d[a, n0:n0 + 8].double().T @ x[a, k0:k0 + 8].double()
            got = grad[e, n0:n0 + 8, k0:k0 + 8].double()
            assert (got - want).abs().max() <= 4 * 2.0 ** -22 * 20 * 25
    assert buf.get_status() == 0


def test_refusals():
    from combine_moonep_plan_gb300._lib import MoonepError
    buf = _buffer(1, 2, 1, 64)
    x, d = (torch.zeros(64, c, device="cuda").bfloat16() for c in (16, 8))
    cu = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    assert buf.NvS == 64
    ok = buf.expert_weight_grad(x, d, cu)
    assert not ok[0].any() and not ok[1].any()
    with pytest.raises(TypeError):
        buf.expert_weight_grad(x.float(), d, cu)
    with pytest.raises(ValueError):
        buf.expert_weight_grad(x[:63], d, cu)
    with pytest.raises(ValueError):
        buf.expert_weight_grad(x, d[:, :7], cu)
    with pytest.raises(ValueError):
        buf.expert_weight_grad(x, d, cu, accumulate=True)
    with pytest.raises(ValueError):
        buf.expert_weight_grad(x, d, cu, out=(ok[0], ok[1][:, :0]))
    with pytest.raises(ValueError):
        buf.expert_weight_grad(x.t().contiguous().t(), d, cu)
    with pytest.raises(MoonepError):   # rows 34 bytes apart
        buf.expert_weight_grad(torch.zeros(64, 17, device="cuda").bfloat16()[:, :16], d, cu)
    with pytest.raises(MoonepError):   # a base off 16 bytes
        buf.expert_weight_grad(torch.zeros(64, 24, device="cuda").bfloat16()[:, 1:17], d, cu)
    assert buf.get_status() == 0
