"""The weight gradients' barrier protocol, on the CPU: the model of
tests/weight_grad_model.py runs clean with the kernel's constants, and finds the
mistakes that are planted in it."""
import pytest

from tests import weight_grad_model as model

# rows of a pair's tiles: none, less than a step, ragged and whole stages, more
# stages than the ring and more than a part, many tiles of several batches
SHAPES = [[1], [0, 0, 0], [64, 64], [65, 0, 15, 16, 17, 0, 63], [7] * 40, [0] * 70,
          [2000, 1, 333], [512, 513, 511, 1024], [16, 80, 320, 321] * 12, [130] * 33,
          [5, 0] * 50, [700, 64, 0, 33] * 17]


def fault(tiles, seed, clear=True, **changed):
    try:
        model.run(dict(model.constants(), **changed), tiles, seed, clear)
    except model.Fault as e:
        return str(e)
    return None


@pytest.mark.parametrize("tiles", SHAPES, ids=lambda t: "%dx%d" % (len(t), max(t)))
def test_kernel_constants(tiles):
    for seed in range(6):
        assert fault(tiles, seed) is None


def found(seeds=8, **kw):
    return {fault(t, s, **kw) for t in SHAPES for s in range(seeds)} - {None}


def test_constants_are_read():
    c = model.constants()
    assert c["full"] == 2 and c["acc_empty"] == 2 * c["kEpilogueWarps"] and c["drain"]
    assert c["kStages"] >= 2 and c["kDeep"] % 16 == 0


def test_finds_wrong_arrival_counts():
    assert any("too many" in f or "another stage" in f or "late" in f or "deadlock" in f
               for f in found(full=1))
    assert any(f.startswith("deadlock") for f in found(full=3))
    assert any("accumulator" in f for f in found(acc_empty=1))
    assert any(f.startswith("deadlock") for f in found(acc_empty=17))
    assert any(f.startswith(("tiles", "deadlock", "too many", "tile of")) for f in
               found(kTileReaders=8))


def test_finds_rows_that_are_not_cleared_in_time():
    assert "rows not cleared" in found(clear=False)


def test_finds_releases_after_a_cta_has_left():
    assert any(f.startswith("late arrival at empty") for f in found(drain=False))
