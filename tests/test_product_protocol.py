"""The expert product's barrier protocol, on the CPU: the model of
tests/product_model.py runs clean with the kernel's constants, and finds the
mistakes that are planted in it."""
import pytest

from tests import product_model as model

# tiles of a pair, stages of a tile: one stage, odd and even counts, fewer and
# more than the ring's stages, one to several batches of tiles
SHAPES = [(1, 1), (2, 6), (3, 28), (5, 14), (35, 2), (38, 6), (40, 1), (70, 5), (97, 3), (130, 1)]


def fault(tiles, stages, seed, ring=0, **changed):
    try:
        model.run(dict(model.constants(), **changed), tiles, stages, seed, ring)
    except model.Fault as e:
        return str(e)
    return None


@pytest.mark.parametrize("tiles,stages", SHAPES)
def test_kernel_constants(tiles, stages):
    for seed in range(4):
        assert fault(tiles, stages, seed) is None


def any_fault(shapes, seeds=12, **kw):
    found = {fault(*s, seed, **kw) for s in shapes for seed in range(seeds)}
    return found - {None}


def test_finds_waits_that_rely_on_the_releases_order():
    """A scale warp that waits for its own stages' releases sees one phase of a
    barrier in two or three, and relies on releases to arrive in order."""
    assert any_fault([(5, 14), (20, 3)], scales_wait="empty") & {"operand overwritten",
                                                                 "operand of another stage"}


def test_finds_a_stage_ring_too_short_for_the_turns():
    shapes = [(5, 14), (20, 3)]
    assert any_fault(shapes, kStages=2) & {"operand overwritten", "operand of another stage"}
    assert not any_fault(shapes, kStages=3)


def test_finds_a_shared_ring_of_boxes():
    """Two sets that share three boxes: a set takes the parity of a use that
    the other set has still to finish for its own."""
    shapes = [(5, 14), (38, 6)]
    assert "scales of another chunk" in any_fault(shapes, ring=3)
    assert not any_fault(shapes, ring=2)     # two boxes are one for each set


@pytest.mark.parametrize("name", ["kFullArrivals", "kAccReaders"])
@pytest.mark.parametrize("by", [-1, 1])
def test_finds_wrong_counts(name, by):
    count = model.constants()[name]
    assert any_fault([(70, 2)], seeds=4, **{name: count + by})


def test_finds_releases_that_outlive_a_cta():
    """The last products release their stages in both CTAs some time after the
    accumulator is announced: a CTA that does not wait for them may be gone."""
    found = any_fault([(1, 1), (2, 6), (5, 14)], drain=False)
    assert found and all(f.startswith("late arrival at empty") for f in found)
