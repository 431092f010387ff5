"""Which tensors the binding takes as sharing memory (an output given by the caller must not overlap an input)."""

import pytest

torch = pytest.importorskip("torch")

import rope_cu_tile_gb300 as pk  # noqa: E402


def elements(t):
    """The storage indexes of a tensor's elements."""
    base = torch.arange(t.untyped_storage().nbytes() // t.element_size())
    return set(base.as_strided(t.shape, t.stride(), t.storage_offset()).flatten().tolist())


VIEWS = [((3, 4), (16, 1), 0), ((3, 4), (16, 1), 4), ((3, 4), (16, 1), 12), ((3, 4), (16, 1), 14), ((3, 8), (16, 1), 2),
         ((1, 8), (8, 1), 0), ((1, 8), (0, 1), 0), ((1, 8), (0, 1), 4), ((1, 8), (0, 1), 8), ((1, 8), (3, 1), 5), ((2, 16), (16, 1), 30),
         ((1, 1), (0, 0), 7), ((0, 8), (8, 1), 0), ((5,), (1,), 3), ((3, 1), (16, 5), 4)]


@pytest.mark.parametrize("a", VIEWS)
@pytest.mark.parametrize("b", VIEWS)
def test_overlap(a, b):
    """Never disjoint where an element is shared; and slices of different columns of one matrix are not taken as sharing."""
    base = torch.zeros(64)
    u, v = base.as_strided(*a), base.as_strided(*b)
    shared = bool(elements(u) & elements(v))
    assert pk._overlap(u, v) or not shared
    if a[0] == b[0] == (3, 4) and not shared:
        assert not pk._overlap(u, v) or {a[2], b[2]} & {14}  # (columns 14 to 17 run into the next row)


def test_rows_of_no_stride():
    """A single row may have any stride, zero among them."""
    base = torch.zeros(64)
    a, b = base.as_strided((1, 8), (0, 1), 0), base.as_strided((1, 8), (0, 1), 4)
    assert pk._overlap(a, b) and pk._overlap(b, a) and not pk._overlap(a, base.as_strided((1, 8), (0, 1), 8))
    with pytest.raises(ValueError, match="out overlaps an input"):
        pk._disjoint(a, "out", b)
