"""num_sms on the router and the expert stage: every launch of a capped Buffer
has no more blocks than that many SMs hold (at least one for every rank, and one
pair of SMs for the product), read from a captured graph; results are those of
an uncapped Buffer."""
import ctypes

import numpy as np
import pytest
import torch

from combine_moonep_plan_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


class _Kernel(ctypes.Structure):
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3),
                ("block", ctypes.c_uint * 3), ("smem", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


def _launches(call):
    """(blocks, blocks that an SM holds) of every kernel that `call` launches;
    captured, not run."""
    cu = ctypes.CDLL("libcuda.so.1")
    ok = lambda e: pytest.fail("driver error %d" % e) if e else None  # noqa: E731
    call()                                       # outputs' memory is in the allocator's cache
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = ctypes.c_void_p()
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        st = ctypes.c_void_p(side.cuda_stream)
        ok(cu.cuStreamBeginCapture_v2(st, 2))
        try:
            call()
        finally:
            ok(cu.cuStreamEndCapture(st, ctypes.byref(graph)))
    n = ctypes.c_size_t(0)
    ok(cu.cuGraphGetNodes(graph, None, ctypes.byref(n)))
    nodes = (ctypes.c_void_p * n.value)()
    ok(cu.cuGraphGetNodes(graph, nodes, ctypes.byref(n)))
    out = []
    for node in nodes:
        kind = ctypes.c_int()
        ok(cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)))
        if kind.value != 0:
            continue
        k = _Kernel()
        ok(cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(k)))
        per = ctypes.c_int()
        ok(cu.cuOccupancyMaxActiveBlocksPerMultiprocessor(
            ctypes.byref(per), ctypes.c_void_p(k.func or k.kern),
            int(np.prod(list(k.block))), ctypes.c_size_t(k.smem)))
        out.append((int(np.prod(list(k.grid))), per.value))
    ok(cu.cuGraphDestroy(graph))
    return out


@pytest.mark.parametrize("num_sms", [1, 6, 40])
def test_blocks_stay_within_the_cap(num_sms):
    from combine_moonep_plan_gb300 import Buffer
    R, S, K, tp, F = 4, 2048, 2, 16, 256
    for E in (8, 24, 48, 128, 200, 300, 500, 640):
        z = torch.randn(R, S, E, device="cuda")
        B = E // R                               # slots enough for any plan
        kw = dict(S=S, H=32, K=K, E=E, num_ep_ranks=R, B=B, token_padding=tp,
                  zero_copy_views=False)
        buf, free = Buffer(num_sms=num_sms, **kw), Buffer(**kw)
        got, want = buf.route(z, balance=0.1), free.route(z, balance=0.1)
        assert torch.equal(got.topk, want.topk) and torch.equal(got.weights, want.weights)
        dw = torch.randn(R, S, K, device="cuda")
        one = torch.ones(1, device="cuda")
        assert torch.allclose(buf.route_backward(got, z, dw, one),
                              free.route_backward(want, z, dw, one), rtol=1e-5, atol=1e-9)
        dz = torch.empty_like(z)
        for call, n in ((lambda: buf.route(z, balance=0.1), 2), (lambda: buf.route(z), 1),
                        (lambda: buf.route_backward(got, z, dw, one, out=dz), 1)):
            launches = _launches(call)
            assert n <= len(launches) <= 2
            # the sums of the loss and of several clusters: one cluster of eight
            for blocks, per in launches[:1]:
                assert blocks <= max(R, num_sms * per), (E, blocks, per)
    topk, _ = wl.routing(wl.Shape("t", R=R, E=E, K=K, S=S, H=32, Hp=32, B=B, tp=tp,
                                  weights="softmax"), "zipf", zipf_s=0.5, seed=1)
    cu = free.plan(torch.from_numpy(topk).cuda()).cu_seqlens.clone()
    n = R * buf.NvS
    x, up, d = (torch.randn(n, F, device="cuda").bfloat16() for _ in range(3))
    w = torch.rand(n, device="cuda")
    weight = free.quantize_mx(torch.randn(E + R * B, 64, F, device="cuda"))
    used = (torch.arange(buf.NvS, device="cuda")[None, :] < cu[:, -1:]).reshape(-1)
    assert int(used.sum()) >= R * S * K and free.get_status() == 0

    def calls(b):
        x4 = (torch.zeros(n, F // 2, dtype=torch.uint8, device="cuda"),
              torch.zeros(n, F // 32, dtype=torch.uint8, device="cuda"))
        y = torch.zeros(n, 64, device="cuda")
        act, back = torch.zeros_like(x), torch.zeros_like(x)
        dg, du, dwn = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w)
        _, ckpt = b.gated_act(x, up, cu, w, checkpoint=True, out=act)
        none = (torch.zeros(n, 0, dtype=torch.uint8, device="cuda"),) * 2
        wnone = (torch.zeros(E + R * B, 64, 0, dtype=torch.uint8, device="cuda"),) * 2
        return [(lambda: b.quantize_mx(x, cu_seqlens=cu, out=x4), x4[0]),
                (lambda: b.quantize_mx(x, out=x4), x4[0]),
                (lambda: b.quantize_mx(x.float(), out=x4), x4[1]),
                (lambda: b.dequantize_mx(*x4, out=back), back),
                (lambda: b.gated_act(x, up, cu, w, out=act), act),
                (lambda: b.gated_act_backward(ckpt, d, cu, w, out=(dg, du, dwn)), dg),
                (lambda: b.expert_product(x4, weight, cu, out=y), y),
                (lambda: b.expert_product(none, wnone, cu, out=y), y)]

    for i, ((call, out), (call0, out0)) in enumerate(zip(calls(buf), calls(free))):
        call()
        call0()
        assert torch.equal(out[used], out0[used]), i
        blocks, per = _launches(call)[-1]        # past a conversion of the input, if any
        assert blocks <= max(R, 2, num_sms * per), (i, blocks, per)
    # what a block's warps do also depends on the rows: few of them
    small = Buffer(S=2, H=32, K=1, E=4, num_ep_ranks=4, B=0, token_padding=1, num_sms=num_sms,
                   zero_copy_views=False)
    cu = torch.full((4, 4), 2, dtype=torch.int32, device="cuda")
    x = torch.randn(8, 4096, device="cuda").bfloat16()
    act = torch.empty_like(x)
    blocks, per = _launches(lambda: small.gated_act(x, x, cu, out=act))[-1]
    assert blocks <= max(4, num_sms * per)
    assert buf.get_status() == 0 and free.get_status() == 0
