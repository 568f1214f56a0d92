"""Microscaled 4-bit tensors, the experts' product and the gated activation
with its 8-bit checkpoint, on the GPU, against 64-bit forms.

Codes and scales are compared exactly.  Products of 4-bit values are exact, so
a product's error is its summation's: at most one part in 2^22 of the sum of
magnitudes for each 32 terms.  The activation's fp32 steps each err by a few
2^-24, and its exponential by |g| 2^-24 more; bf16 outputs add half of 2^-8.
"""
import numpy as np
import pytest
import torch

from combine_moonep_plan_gb300 import workloads as wl
from tests import expert_refs as ref

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -23
BF16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def _buffer(R, S, K, E, B, tp, **kw):
    from combine_moonep_plan_gb300 import Buffer
    return Buffer(S=S, H=32, K=K, E=E, num_ep_ranks=R, B=B, token_padding=tp,
                  zero_copy_views=False, **kw)


def _planned(R, S, K, E, B, tp, zipf, seed):
    """(Buffer, cu_seqlens on the device, on the host) of a real plan."""
    sh = wl.Shape("t", R=R, E=E, K=K, S=S, H=32, Hp=32, B=B, tp=tp, weights="softmax")
    topk, _ = wl.routing(sh, "zipf", zipf_s=zipf, seed=seed)
    buf = _buffer(R, S, K, E, B, tp)
    plan = buf.plan(torch.from_numpy(topk).cuda())
    assert buf.get_status() == 0
    return buf, plan.cu_seqlens.clone(), plan.cu_seqlens.cpu().numpy()


def _rows_mask(cu, NvS):
    return (np.arange(NvS)[None, :] < cu[:, -1:]).reshape(-1)


# ------------------------------------------------------------------ formats

def _values(rows, cols, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)) * 4)
    edge = [0.0, -0.0, 1e-39, -1e-45, 3e38, 6.0, 7.9, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0,
            -0.25, -5.0, 2.0 ** -126, 2.0 ** -127, 448.0, 464.0, 480.0, 496.0]
    n = min(rows * cols, len(edge) * 7)
    flat = x.reshape(-1)
    flat[:n] = np.resize(edge, n) * np.repeat([1, 2.0 ** -20, 1, 1, 1, 1, 1], len(edge))[:n]
    if rows > 4:
        x[2] = 0.0
        x[3, ::5] = 2.0 ** -130
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (7, 1184), (5, 4096), (1000, 64),
                                       (33, 7168)])
def test_quantise_and_read_back(rows, cols, dtype):
    x = torch.from_numpy(_values(rows, cols, rows + cols)).to(dtype).cuda()
    buf = _buffer(1, 1, 1, 1, 0, 1)
    packed, scales = buf.quantize_mx(x)
    xn = x.float().cpu().numpy().astype(np.float64)
    codes, want_s = ref.mx_encode(xn, ref.E2M1, 2, 8)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    got = ref.unpack(packed.cpu().numpy())
    back = ref.mx_decode(got, want_s, ref.E2M1, 8)
    assert np.array_equal(back, ref.mx_decode(codes, want_s, ref.E2M1, 8))
    for t in (torch.float32, torch.bfloat16):
        y = buf.dequantize_mx(packed, scales, dtype=t)
        # every value is one bf16 holds (below 2^-126 as a subnormal)
        assert np.array_equal(y.float().cpu().numpy().astype(np.float64), back)


def test_every_scale_byte_and_code_reads_back():
    buf = _buffer(1, 1, 1, 1, 0, 1)
    packed = torch.arange(256, dtype=torch.uint8, device="cuda").repeat_interleave(16)
    packed = (packed.view(256, 16) + 16 * torch.arange(16, device="cuda", dtype=torch.uint8) +
              torch.arange(16, device="cuda", dtype=torch.uint8)).contiguous()
    scales = torch.arange(256, dtype=torch.uint8, device="cuda").view(256, 1)
    y = buf.dequantize_mx(packed, scales, dtype=torch.float32).cpu().numpy()
    want = ref.mx_decode(ref.unpack(packed.cpu().numpy()), scales.cpu().numpy(), ref.E2M1, 8)
    with np.errstate(over="ignore"):
        assert np.array_equal(y, want.astype(np.float32), equal_nan=True)


def test_non_finite_blocks_read_back_as_nan():
    buf = _buffer(1, 1, 1, 1, 0, 1)
    x = torch.randn(4, 96, device="cuda")
    x[0, 5] = float("nan")
    x[1, 40] = float("inf")
    x[2, 95] = -float("inf")
    for t in (torch.float32, torch.bfloat16):
        packed, scales = buf.quantize_mx(x.to(t))
        y = buf.dequantize_mx(packed, scales).float().cpu().numpy().reshape(4, 3, 32)
        bad = np.zeros((4, 3), bool)
        bad[0, 0] = bad[1, 1] = bad[2, 2] = True
        assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()


def test_quantise_leaves_unused_rows():
    buf, cu, cun = _planned(2, 9, 2, 4, 2, 8, 1.0, 3)
    n = 2 * buf.NvS
    x = torch.randn(n, 64, device="cuda").bfloat16()
    out = (torch.full((n, 32), 77, dtype=torch.uint8, device="cuda"),
           torch.full((n, 2), 78, dtype=torch.uint8, device="cuda"))
    buf.quantize_mx(x, cu_seqlens=cu, out=out)
    used = _rows_mask(cun, buf.NvS)
    assert used.any() and not used.all()
    p, s = buf.quantize_mx(x)
    assert torch.equal(out[0][used], p[used]) and torch.equal(out[1][used], s[used])
    assert (out[0][~used] == 77).all() and (out[1][~used] == 78).all()


# ------------------------------------------------------------------ product

PRODUCTS = [
    # R, S, K, E, B, tp, zipf, N, Kd
    (1, 1, 1, 1, 0, 1, 0.0, 8, 32),
    (1, 1, 1, 1, 1, 1, 0.0, 128, 64),
    (2, 3, 2, 4, 2, 1, 1.5, 40, 96),
    (2, 64, 2, 8, 4, 8, 1.2, 128, 256),
    (3, 50, 2, 21, 3, 1, 1.0, 200, 160),
    (8, 20, 4, 16, 2, 16, 0.5, 264, 544),
    (1, 300, 1, 2, 1, 1, 0.3, 1000, 1184),
    (4, 130, 2, 4, 1, 128, 2.0, 520, 512),
    (8, 128, 8, 128, 16, 16, 1.0, 256, 1536),
    (2, 700, 2, 2, 1, 1, 0.0, 776, 1056),
]


def _weights(G, N, Kd, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randint(0, 256, (G, N, Kd // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.randint(118, 130, (G, N, Kd // 32), generator=g, device="cuda", dtype=torch.uint8)
    return w, s


def _decoded(packed, scales):
    """fp64 values on the device."""
    table = torch.from_numpy(np.concatenate((ref.E2M1, -ref.E2M1))).cuda()
    codes = torch.stack((packed & 15, packed >> 4), -1).reshape(*packed.shape[:-1], -1)
    two = torch.from_numpy(np.ldexp(1.0, np.arange(256) - 127)).cuda()
    two[255] = float("nan")
    v = table[codes.long()].reshape(*scales.shape, 32) * two[scales.long()][..., None]
    return v.reshape(*packed.shape[:-1], -1)


def _check_product(out, rows, weight, cun, E, R, B, NvS, poison):
    a, w = _decoded(*rows), weight
    used = torch.zeros(out.shape[0], dtype=torch.bool, device="cuda")
    Kd = a.shape[1]
    for g, first, n in ref.segments(cun, E, R, B, NvS):
        x = a[first:first + n]
        y = _decoded(w[0][g], w[1][g])
        want, mag = x @ y.T, x.abs() @ y.abs().T
        got = out[first:first + n].double()
        tol = (Kd // 32 + 2) * 2.0 ** -22 * mag
        if out.dtype == torch.bfloat16:
            tol = tol + want.abs() * BF16
        assert bool(((got - want).abs() <= tol).all()), (g, float((got - want).abs().max()))
        used[first:first + n] = True
    assert bool((out[~used] == poison).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,S,K,E,B,tp,zipf,N,Kd", PRODUCTS)
def test_product(R, S, K, E, B, tp, zipf, N, Kd, dtype):
    buf, cu, cun = _planned(R, S, K, E, B, tp, zipf, seed=N + Kd)
    n = R * buf.NvS
    x = torch.randn(n, Kd, device="cuda").bfloat16()
    rows = buf.quantize_mx(x)
    # rows outside every segment may hold anything
    unused = torch.from_numpy(~_rows_mask(cun, buf.NvS)).cuda()
    rows[0][unused] = 0x7f
    rows[1][unused] = 255
    weight = _weights(E + R * B, N, Kd, 1)
    out = torch.full((n, N), 5.0, dtype=dtype, device="cuda")
    buf.expert_product(rows, weight, cu, out=out)
    _check_product(out, rows, weight, cun, E, R, B, buf.NvS, 5.0)
    assert buf.get_status() == 0


@pytest.mark.parametrize("num_sms,R,S,K,E,B,tp,N,Kd", [
    (2, 8, 128, 8, 128, 16, 16, 512, 512),      # one pair of SMs: hundreds of tiles in a row
    (2, 2, 300, 2, 4, 2, 1, 4096, 96),          # one stage per tile
    (5, 8, 64, 4, 64, 8, 8, 1024, 1184),        # odd count of stages, scales not in vectors
    (6, 1, 40, 4, 1100, 7, 1, 16, 64),          # more groups than the tile table has entries
    (None, 8, 64, 8, 128, 16, 1, 8192, 64),     # more tiles than two batches of the schedule
])
def test_product_long_tile_sequences(num_sms, R, S, K, E, B, tp, N, Kd):
    from combine_moonep_plan_gb300 import Buffer
    sh = wl.Shape("t", R=R, E=E, K=K, S=S, H=32, Hp=32, B=B, tp=tp, weights="softmax")
    topk, _ = wl.routing(sh, "zipf", zipf_s=0.8, seed=N)
    buf = Buffer(S=S, H=32, K=K, E=E, num_ep_ranks=R, B=B, token_padding=tp, num_sms=num_sms,
                 zero_copy_views=False)
    cu = buf.plan(torch.from_numpy(topk).cuda()).cu_seqlens.clone()
    n = R * buf.NvS
    rows = buf.quantize_mx(torch.randn(n, Kd, device="cuda"))
    weight = _weights(E + R * B, N, Kd, 4)
    out = torch.full((n, N), 5.0, device="cuda")
    for _ in range(3):                           # back to back: launches overlap their starts
        buf.expert_product(rows, weight, cu, out=out)
    _check_product(out, rows, weight, cu.cpu().numpy(), E, R, B, buf.NvS, 5.0)
    assert buf.get_status() == 0


def test_product_of_spaced_rows():
    """Rows that lie apart: codes and scales of a row in one record, the form
    a plan can dispatch in one copy."""
    R, S, K, E, B, tp, N, Kd = 2, 40, 2, 4, 2, 8, 136, 1024
    buf, cu, cun = _planned(R, S, K, E, B, tp, 1.0, 4)
    n = R * buf.NvS
    packed, scales = buf.quantize_mx(torch.randn(n, Kd, device="cuda"))
    record = torch.cat((packed, scales), 1)
    assert record.shape[1] % 16 == 0
    rows = (record[:, :Kd // 2], record[:, Kd // 2:])
    weight = _weights(E + R * B, N, Kd, 2)
    dense = buf.expert_product((packed, scales), weight, cu, out=torch.zeros(
        n, N, device="cuda"))
    spaced = buf.expert_product(rows, weight, cu, out=torch.zeros(n, N, device="cuda"))
    assert torch.equal(dense, spaced)
    _check_product(spaced, (packed, scales), weight, cun, E, R, B, buf.NvS, 0.0)


def test_product_nan_scale_reaches_its_own_outputs_only():
    buf, cu, cun = _planned(1, 40, 1, 2, 0, 1, 0.0, 5)
    n, N, Kd = buf.NvS, 64, 320
    rows = buf.quantize_mx(torch.randn(n, Kd, device="cuda"))
    w, ws = _weights(2, N, Kd, 3)
    rows[1][3, 2] = 255
    ws[1, 7, 4] = 255
    out = buf.expert_product(rows, (w, ws), cu, out=torch.zeros(n, N, device="cuda"))
    want = torch.zeros(n, N, dtype=torch.bool)
    want[3] = True
    want[int(cun[0, 0]):int(cun[0, 1]), 7] = True
    assert torch.equal(out.isnan().cpu(), want)


def test_product_no_terms_gives_zeros_and_no_rows_nothing():
    buf, cu, cun = _planned(1, 10, 1, 2, 1, 1, 0.0, 6)
    n = buf.NvS
    out = torch.full((n, 16), 3.0, device="cuda")
    e = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    buf.expert_product((e(n, 0), e(n, 0)), (e(3, 16, 0), e(3, 16, 0)), cu, out=out)
    used = torch.from_numpy(_rows_mask(cun, n)).cuda()
    assert (out[used] == 0).all() and (out[~used] == 3).all()
    out.fill_(3.0)
    buf.expert_product((e(n, 16), e(n, 1)), (e(3, 16, 16), e(3, 16, 1)),
                       torch.zeros_like(cu), out=out)
    assert (out == 3).all()


def test_product_reports_offsets_outside_the_window():
    from combine_moonep_plan_gb300 import _lib
    buf, cu, cun = _planned(2, 10, 1, 2, 1, 1, 0.0, 7)
    n, N, Kd = 2 * buf.NvS, 16, 64
    rows = buf.quantize_mx(torch.randn(n, Kd, device="cuda"))
    w = _weights(4, N, Kd, 3)
    for x, v in ((0, -5), (0, buf.NvS + 1), (2, 1 << 30)):
        bad = cu.clone()
        bad[0, x] = v
        out = torch.full((n, N), 3.0, device="cuda")
        buf.expert_product(rows, w, bad, out=out)
        assert buf.get_status() == _lib.ERR_PLAN
        good = torch.full((n, N), 3.0, device="cuda")
        buf.expert_product(rows, w, cu, out=good)
        assert buf.get_status() == 0
        # the other rank's rows are as ever
        assert torch.equal(out[buf.NvS:], good[buf.NvS:])


def test_product_refusals():
    from combine_moonep_plan_gb300._lib import MoonepError
    buf, cu, _ = _planned(1, 10, 1, 2, 1, 1, 0.0, 8)
    n = buf.NvS
    rows = buf.quantize_mx(torch.randn(n, 64, device="cuda"))
    w = _weights(3, 16, 64, 1)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    with pytest.raises(ValueError):
        buf.expert_product(rows, (w[0][:2], w[1]), cu)              # a weight row short
    with pytest.raises(ValueError):
        buf.expert_product(rows, (u8(3, 12, 32), u8(3, 12, 2)), cu)  # N not a multiple of 8
    with pytest.raises(ValueError):
        buf.expert_product((rows[0][:, :16], rows[1]), w, cu)
    with pytest.raises(TypeError):
        buf.expert_product(rows, (w[0].int(), w[1]), cu)
    with pytest.raises(TypeError):
        buf.expert_product(rows, w, cu, dtype=torch.float16)
    with pytest.raises(ValueError):
        buf.expert_product(rows, w, cu[:, :2])
    wide = u8(n, 40)[:, :32]                                         # rows 40 bytes apart
    with pytest.raises(MoonepError):
        buf.expert_product((wide, rows[1]), w, cu)
    with pytest.raises(ValueError):
        buf.expert_product((u8(32, n).t(), rows[1]), w, cu)
    with pytest.raises(ValueError):
        buf.quantize_mx(torch.randn(4, 48, device="cuda"))
    with pytest.raises(TypeError):
        buf.quantize_mx(torch.zeros(4, 64, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        buf.quantize_mx(torch.zeros(n + 1, 64, device="cuda"), cu_seqlens=cu)
    with pytest.raises(ValueError):
        buf.dequantize_mx(rows[0], u8(n, 3))
    buf.destroy()
    with pytest.raises(MoonepError):
        buf.expert_product(rows, w, cu)


# --------------------------------------------------------------- activation

GATED = [
    # R, S, K, E, B, tp, zipf, F, weighted, scale of gate
    (1, 1, 1, 1, 0, 1, 0.0, 32, True, 1.0),
    (2, 9, 2, 4, 2, 8, 1.0, 96, False, 3.0),
    (3, 50, 2, 21, 3, 1, 1.0, 160, True, 1.0),
    (8, 16, 8, 128, 16, 16, 1.0, 1536, True, 1.0),
    (1, 33, 1, 2, 1, 1, 0.5, 1184, True, 30.0),
    (2, 70, 2, 4, 2, 128, 1.0, 2048, False, 1.0),
]


@pytest.mark.parametrize("R,S,K,E,B,tp,zipf,F,weighted,size", GATED)
def test_gated_act_and_gradient(R, S, K, E, B, tp, zipf, F, weighted, size):
    buf, cu, cun = _planned(R, S, K, E, B, tp, zipf, seed=F)
    n = R * buf.NvS
    used = _rows_mask(cun, buf.NvS)
    bf = lambda s: (torch.randn(n, F, device="cuda") * s).bfloat16()  # noqa: E731
    gate, up, d = bf(size), bf(1.0), bf(0.1)
    gate[:, ::31] = 0.0
    w = torch.rand(n, device="cuda") if weighted else None
    # rows outside every segment may hold anything
    poison = torch.from_numpy(~used).cuda()
    for t in (gate, up, d):
        t[poison] = float("nan")
    if weighted:
        w[poison] = float("nan")
    act = torch.full((n, F), 7.0, dtype=torch.bfloat16, device="cuda")
    buf.gated_act(gate, up, cu, w, out=act)
    f64 = lambda t: t[torch.from_numpy(used).cuda()].double().cpu().numpy()  # noqa: E731
    g, u, dd = f64(gate), f64(up), f64(d)
    ww = f64(w)[:, None] if weighted else 1.0
    want = ref.gated(g, u, ww)
    tol = np.abs(want) * ((np.abs(g) + 16) * EPS + BF16) + 1e-38
    assert np.all(np.abs(f64(act) - want) <= tol)
    assert (act[poison] == 7).all()
    # with a checkpoint: the same result, and exact codes
    act2 = torch.full_like(act, 7.0)
    _, ckpt = buf.gated_act(gate, up, cu, w, checkpoint=True, out=act2)
    assert torch.equal(act, act2)
    sel = torch.from_numpy(used).cuda()
    vals = []
    for codes, scales, x in ((ckpt[0], ckpt[2], g), (ckpt[1], ckpt[3], u)):
        c, s = ref.mx_encode(x, ref.E4M3, 8, 128)
        assert np.array_equal(scales[sel].cpu().numpy(), s)
        got = ref.mx_decode(codes[sel].cpu().numpy(), s, ref.E4M3, 128)
        assert np.array_equal(got, ref.mx_decode(c, s, ref.E4M3, 128))
        vals.append(got)
    g8, u8 = vals
    assert np.all(np.abs(g8 - g) <= np.abs(g).reshape(len(g), -1, 32).max(-1).repeat(32, -1)
                  .reshape(g.shape) * 2.0 ** -3)
    # gradient at the checkpoint's values
    dg = torch.full_like(act, 7.0)
    du = torch.full_like(act, 7.0)
    dw = torch.full((n,), 7.0, device="cuda") if weighted else None
    buf.gated_act_backward(ckpt, d, cu, w, out=(dg, du, dw))
    want_g, want_u, want_w = ref.gated_grad(g8, u8, ww, dd)
    s = ref.sigmoid(g8)
    tol = np.abs(ww * dd * u8) * s * (1 + np.abs(g8)) * (np.abs(g8) + 16) * 2 * EPS \
        + np.abs(want_g) * BF16 + 1e-38
    assert np.all(np.abs(f64(dg) - want_g) <= tol)
    tol = np.abs(want_u) * ((np.abs(g8) + 16) * EPS + BF16) + 1e-38
    assert np.all(np.abs(f64(du) - want_u) <= tol)
    assert (dg[poison] == 7).all() and (du[poison] == 7).all()
    if weighted:
        mag = np.abs(dd * g8 * s * u8)
        tol = (mag * (np.abs(g8) + 16 + F) * EPS).sum(-1) + 1e-38
        assert np.all(np.abs(f64(dw) - want_w) <= tol)
        assert (dw[poison] == 7).all()
    assert buf.get_status() == 0


def test_gated_gradient_against_differences():
    """Central differences of <d, act> in 64 bits at the checkpoint's values;
    step 1e-4: about 1e-8 of truncation; bf16 outputs add 2^-9 relative."""
    buf, cu, cun = _planned(1, 6, 1, 1, 0, 1, 0.0, 2)
    n, F = buf.NvS, 32
    gate, up = (torch.randn(n, F, device="cuda").bfloat16() for _ in range(2))
    d = torch.randn(n, F, device="cuda").bfloat16()
    w = torch.rand(n, device="cuda") + 0.5
    _, ckpt = buf.gated_act(gate, up, cu, w, checkpoint=True)
    dg, du, dw = buf.gated_act_backward(ckpt, d, cu, w)
    dec = lambda c, s: ref.mx_decode(c.cpu().numpy(), s.cpu().numpy(), ref.E4M3, 128)  # noqa: E731
    g, u = dec(ckpt[0], ckpt[2]), dec(ckpt[1], ckpt[3])
    dn, wn = d.double().cpu().numpy(), w.double().cpu().numpy()[:, None]
    h = 1e-4
    num_g = dn * (ref.gated(g + h, u, wn) - ref.gated(g - h, u, wn)) / (2 * h)
    num_u = dn * (ref.gated(g, u + h, wn) - ref.gated(g, u - h, wn)) / (2 * h)
    num_w = (dn * (ref.gated(g, u, wn + h) - ref.gated(g, u, wn - h)) / (2 * h)).sum(1)
    for got, num in ((dg, num_g), (du, num_u)):
        assert np.all(np.abs(got.double().cpu().numpy() - num) <= np.abs(num) * BF16 + 1e-6)
    assert np.all(np.abs(dw.double().cpu().numpy() - num_w) <= 1e-5 * (1 + np.abs(num_w)))


def test_gated_extreme_values():
    """Large and infinite gates: the sigmoid neither overflows nor loses the
    sign; a non-finite block's checkpoint reads as NaN and touches no other."""
    buf, cu, _ = _planned(1, 4, 1, 1, 0, 1, 0.0, 2)
    n, F = buf.NvS, 64
    gate = torch.zeros(n, F, device="cuda").bfloat16()
    gate[0, :6] = torch.tensor([100.0, -100.0, 3e38, -3e38, 80.0, -80.0], device="cuda")
    up = torch.ones_like(gate)
    gate[1, 0] = float("inf")
    gate[2, 1] = float("nan")
    act, ckpt = buf.gated_act(gate, up, cu, checkpoint=True)
    a = act.float().cpu().numpy()
    assert np.array_equal(a[0, :3], gate[0, :3].float().cpu().numpy() * [1, 0, 1]) or \
        (a[0, 0] == 100 and abs(a[0, 1]) < 1e-38 and a[0, 2] > 2.9e38)
    assert a[0, 3] == 0 and abs(a[0, 5]) < 1e-30
    assert np.isposinf(a[1, 0]) and np.isnan(a[2, 1])
    assert np.isfinite(a[1, 1:]).all() and np.isfinite(np.delete(a[2], 1)).all()
    dg, du, _ = buf.gated_act_backward(ckpt, torch.ones_like(gate), cu)
    for t in (dg, du):
        t = t.float().cpu().numpy()
        assert np.isfinite(t[0]).all() and np.isfinite(t[3]).all()
        assert np.isnan(t[1, :32]).all() and np.isfinite(t[1, 32:]).all()
        assert np.isnan(t[2, :32]).all() and np.isfinite(t[2, 32:]).all()


def test_gated_refusals():
    from combine_moonep_plan_gb300._lib import MoonepError
    buf, cu, _ = _planned(1, 4, 1, 1, 0, 1, 0.0, 2)
    n = buf.NvS
    z = torch.zeros(n, 64, device="cuda").bfloat16()
    with pytest.raises(TypeError):
        buf.gated_act(z.float(), z.float(), cu)
    with pytest.raises(ValueError):
        buf.gated_act(z, z[:, :32], cu)
    with pytest.raises(ValueError):
        buf.gated_act(z[:, :32], z[:, :32], cu)               # not contiguous
    odd = torch.zeros(n, 40, device="cuda").bfloat16()
    with pytest.raises(ValueError):
        buf.gated_act(odd, odd, cu)
    with pytest.raises(TypeError):
        buf.gated_act(z, z, cu.long())
    with pytest.raises(ValueError):
        buf.gated_act(z, z, cu, torch.zeros(n + 1, device="cuda"))
    _, ckpt = buf.gated_act(z, z, cu, checkpoint=True)
    with pytest.raises(ValueError):
        buf.gated_act_backward(ckpt[:3], z, cu)
    with pytest.raises(ValueError):
        buf.gated_act_backward((ckpt[0], ckpt[1], ckpt[2], ckpt[3][:, :1]), z, cu)
    buf.destroy()
    with pytest.raises(MoonepError):
        buf.gated_act(z, z, cu)
