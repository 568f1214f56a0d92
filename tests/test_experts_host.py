"""Host-side refusals of the router's and the expert stage's entry points: a
missing context or a bad argument returns at once, with nothing launched."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from combine_moonep_plan_gb300 import build
    build.build()
    from combine_moonep_plan_gb300 import _lib
    return _lib.load()


def test_null_context_refused(lib):
    from combine_moonep_plan_gb300._lib import ERR_INVALID_ARG
    n = None
    assert lib.moonep_route(n, n, 0, 0, 0.0, 0, n, n, n, n, n, n, n) == ERR_INVALID_ARG
    assert lib.moonep_route_backward(n, n, 0, 0, n, n, n, n, n, n, n, n) == ERR_INVALID_ARG
    assert lib.moonep_quantize_mx(n, n, 0, 1, 32, n, n, n, n) == ERR_INVALID_ARG
    assert lib.moonep_dequantize_mx(n, n, n, 0, 1, 32, n, n) == ERR_INVALID_ARG
    assert lib.moonep_expert_product(n, n, n, 16, n, 1, n, n, 8, 32, 0, n, n) == ERR_INVALID_ARG
    assert lib.moonep_gated_act(n, n, n, n, n, 32, n, n, n, n, n, n) == ERR_INVALID_ARG
    assert lib.moonep_gated_act_backward(n, n, n, n, n, n, n, n, 32, n, n, n, n) == \
        ERR_INVALID_ARG


def test_package_exports():
    import combine_moonep_plan_gb300 as pkg
    assert pkg.Route.__name__ == "Route" and pkg.GatedCheckpoint.__name__ == "GatedCheckpoint"
    with pytest.raises(AttributeError):
        pkg.Router
