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
