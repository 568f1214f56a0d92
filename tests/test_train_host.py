"""Host-side refusals and layouts of the training operators: a missing context or a
bad argument returns at once, with nothing launched; no GPU needed."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    from combine_moonep_plan_gb300 import _lib
    return _lib.load()


def test_null_context_refused(lib):
    from combine_moonep_plan_gb300 import _lib
    bad, n = _lib.ERR_INVALID_ARG, None
    sel = ctypes.byref(_lib.MoonepRouteSelection(None, 1, 1, 0, 1, 1.0))
    cfg = ctypes.byref(_lib.MoonepAdamwConfig(lr=1, beta1=.9, beta2=.9, eps=1, step=1, bits=32))
    assert lib.moonep_route_select(n, n, 0, 0, sel, 0.0, 0, n, n, n, n, n, n, n) == bad
    assert lib.moonep_route_select_backward(n, n, 0, 0, sel, n, n, n, n, n, n, n, n) == bad
    assert lib.moonep_update_route_bias(n, n, n, 0.0, n, n) == bad
    assert lib.moonep_expert_weight_grad(n, n, n, 16, n, 16, 8, 8, 0, n, n, n, n) == bad
    assert lib.moonep_expert_weight_grad_workspace(n, 8, 8) == 0
    assert lib.moonep_grad_norm_workspace(n) == 0
    assert lib.moonep_grad_norm(n, 0, n, n, 0, n, n, n) == bad
    assert lib.moonep_adamw(n, cfg, 0, n, n, n, n, n, n, n, n, n) == bad
    assert lib.moonep_adamw_moments(n, 32, n, n, n, n, 0, n, n, n) == bad


def test_structures_as_the_header_lays_them_out():
    from combine_moonep_plan_gb300 import _lib
    assert ctypes.sizeof(_lib.MoonepRouteSelection) == 32
    assert ctypes.sizeof(_lib.MoonepAdamwConfig) == 5 * 8 + 3 * 8 + 7 * 4 + 4


def test_state_layout():
    from combine_moonep_plan_gb300.api import AdamWState
    sizes = [1, 0, 32, 33, 100]
    for bits in (32, 8):
        s = AdamWState(None, sizes, bits, "cpu")
        assert s.offsets == [0, 32, 32, 64, 128] and s.total == 256
        parts = s.split(s.tensors[0])
        assert [p.numel() for p in parts] == sizes
        m, v, ms, vs = s._pointers()
        base = s.tensors[0].data_ptr()
        step = 4 if bits == 32 else 1
        assert [p - base for p in m] == [step * o for o in s.offsets]
        if bits == 8:
            assert [t.numel() for t in s.tensors] == [256, 8, 256, 8]
            assert [p - s.tensors[1].data_ptr() for p in ms] == [o // 32 for o in s.offsets]
            assert [p - s.tensors[2].data_ptr() for p in v] == s.offsets
        else:
            assert ms is None and vs is None
        # moments that moved are found again
        s.tensors = tuple(t.clone() for t in s.tensors)
        assert s._pointers()[0][0] == s.tensors[0].data_ptr()


def test_lists_are_checked():
    from combine_moonep_plan_gb300.api import _FLOATS, _check_bf16_rows, _check_list
    cpu = torch.zeros(4)
    with pytest.raises(ValueError):
        _check_list([cpu], "x", _FLOATS, None)
    with pytest.raises(TypeError):
        _check_list([cpu.half()], "x", _FLOATS, None)
    with pytest.raises(TypeError):
        _check_list([cpu, cpu.bfloat16()], "x", _FLOATS, None)
    with pytest.raises(ValueError):
        _check_list([cpu], "x", _FLOATS, (3,))
    with pytest.raises(ValueError):
        _check_list([cpu], "x", _FLOATS, (4, 4))
    assert _check_list([], "x", _FLOATS, None) == (torch.float32, [], [])
    with pytest.raises(ValueError):
        _check_bf16_rows(torch.zeros(4, 8, dtype=torch.bfloat16), "x", 4)


def test_package_exports():
    import combine_moonep_plan_gb300 as pkg
    assert pkg.AdamWState.__name__ == "AdamWState"
