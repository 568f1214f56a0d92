"""How exact long sums of the experts' weight gradients are.

With terms of one sign the result is the sum of the terms' magnitudes.  A sum on the
tensor cores takes 16 rows at a time, each addition off by at most 2^-22 of it (see
test_gpu_weight_grad.py), and ends after 512 rows: (512 / 16 + 2) 2^-22.  The parts
are added up in fp32, 2^-24 of the result each; shares of a segment only make these
additions fewer one after another.  An unbroken sum over n rows drops bits at each of
its n / 16 additions, always downwards.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


@pytest.mark.parametrize("N,Kd,shares", [(2048, 2048, False), (128, 256, True)])
@pytest.mark.parametrize("rows", [2048, 60000])
def test_long_sums_of_one_sign(N, Kd, shares, rows):
    from combine_moonep_plan_gb300 import Buffer, _lib
    buf = Buffer(S=2 * rows, H=8, K=1, E=2, num_ep_ranks=1, B=0, token_padding=1,
                 zero_copy_views=False)
    assert (_lib.load().moonep_expert_weight_grad_workspace(buf._ctx, N, Kd) > 0) == shares
    g = torch.Generator(device="cuda").manual_seed(rows + N)
    x, d = (torch.rand(buf.NvS, c, generator=g, device="cuda").bfloat16() for c in (Kd, N))
    cu = torch.tensor([[rows, 2 * rows - 5]], dtype=torch.int32, device="cuda")
    grad, _ = buf.expert_weight_grad(x, d, cu)
    tol = (512 / 16 + 2) * 2.0 ** -22 + (rows / 512 + 1) * 2.0 ** -24
    for e, a in enumerate((slice(0, rows), slice(rows, 2 * rows - 5))):
        want = d[a, :64].double().T @ x[a, -96:].double()
        off = (grad[e, :64, -96:].double() - want).abs() / want
        assert off.max().item() <= tol
    assert buf.get_status() == 0
