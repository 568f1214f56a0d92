"""Host-side checks of the optimizer's lists and moments; no GPU needed."""
import pytest
import torch


def _state(bits, sizes=(1, 0, 33, 100)):
    from combine_moonep_plan_gb300.api import AdamWState
    return AdamWState(None, list(sizes), bits, "cpu")


@pytest.mark.parametrize("bits", [32, 8])
def test_replaced_moments_are_looked_at(bits):
    """Moments that were replaced, as by a checkpoint, are taken at their new place
    when they are like the old ones, and refused before their addresses are read
    otherwise."""
    def bad(tensors):
        s = _state(bits)
        s._pointers()
        s.tensors = tensors
        for ask in (s._pointers, s.moments):
            with pytest.raises(ValueError):
                ask()

    have = _state(bits).tensors
    bad(have[:-1])
    bad((*have, have[0]))
    for k in range(len(have)):
        other = lambda t: tuple(t if i == k else h for i, h in enumerate(have))  # noqa: E731
        bad(other(have[k][:-1]))
        bad(other(torch.cat([have[k], have[k]])))
        bad(other(have[k].reshape(1, -1)))
        bad(other(have[k].half()))
        bad(other(have[k].to("meta")))
        bad(other(torch.cat([have[k], have[k]])[::2]))
    s = _state(bits)
    s.tensors = [t.clone() for t in have]
    got = s._pointers()
    assert got[0][0] == s.tensors[0].data_ptr() and s.split(s.tensors[0])[3].numel() == 100


def test_shapes_of_gradients_and_copies():
    from combine_moonep_plan_gb300.api import _check_shapes
    p = [torch.zeros(s) for s in ((4, 6), (24,), (2, 3, 4), ())]
    view = lambda *s: torch.zeros(24).view(*s)  # noqa: E731
    one = torch.zeros(1)
    for good in ([view(4, 6), view(24), view(2, 3, 4), one[0]], [view(24)] * 3 + [one],
                 [view(2, 3, 4), view(4, 6), view(4, 6), one]):
        _check_shapes(good, "grads", p)
    for bad in ([view(6, 4), view(24), view(2, 3, 4), one],
                [view(4, 6), view(24), view(2, 4, 3), one],
                [view(1, 24), view(24), view(2, 3, 4), one]):
        with pytest.raises(ValueError):
            _check_shapes(bad, "grads", p)
    _check_shapes([], "grads", [])
    _check_shapes([view(6, 4)], "grads", [view(24)])


def test_one_device():
    from combine_moonep_plan_gb300.api import _check_one_device
    for places in (set(), {None}, {0}, {None, 1}):
        _check_one_device(places)
    for places in ({0, 1}, {None, 0, 1}, {-1, 0}):
        with pytest.raises(ValueError):
            _check_one_device(places)
