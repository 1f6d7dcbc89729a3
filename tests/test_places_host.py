"""Where the rows of two tensors lie, against sets of their bytes."""

import random

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dsa():
    import deepseek_sparse_attention_row_gb300 as dsa

    return dsa


def rows(place):
    address, row, T, H, st, sh = place
    return [range(address + t * st + h * sh, address + t * st + h * sh + row)
            for t in range(T) for h in range(H)]


def drawn(rng):
    size, D = rng.choice([2, 4]), rng.randint(1, 5)
    T, H = rng.randint(1, 5), rng.randint(1, 4)
    st, sh = rng.choice([(H * D, D), (D, T * D), (2 * H * D, 2 * D), (H * D + 3, D), (3 * D, 7 * D),
                         (rng.randint(0, 20), rng.randint(0, 20)), (H * D, 0), (24, 6)])
    return size, (T, H, D), (st, sh)


@pytest.mark.parametrize("seed", range(8))
def test_places(dsa, seed):
    rng = random.Random(seed)
    seen = [0, 0, 0]
    for _ in range(1500):
        size, shape, strides = drawn(rng)
        a = dsa._place(1000, shape, strides, size)
        size, shape, strides = drawn(rng) if rng.random() < 0.5 else (size, shape, strides)
        b = dsa._place(1000 + rng.randint(-60, 60), shape, strides, size)
        assert dsa._rows_overlap(b) == (len({x for r in rows(b) for x in r})
                                        < sum(map(len, rows(b))))
        inside = {x for r in rows(a) for x in r}
        apart = not any(x in inside for r in rows(b) for x in r)
        assert dsa._apart(a, b) == apart == dsa._apart(b, a), (a, b)
        seen[0] += apart
        seen[1] += not apart
        seen[2] += apart and max(r[0] for r in rows(a)) > b[0] and max(r[0] for r in rows(b)) > a[0]
    assert min(seen) > 50  # apart, not, and apart but interleaved


def test_no_rows(dsa):
    for shape in ((0, 2, 4), (2, 0, 4), (2, 2, 0)):
        assert dsa._place(1000, shape, (8, 4), 2) is None
    assert dsa._place(None, (2, 2, 4), None, 2) is None


A, B = (1000, 8, 4, 2, 32, 8), (1016, 8, 4, 2, 32, 8)  # halves of the same rows
FAR = (9000, 8, 4, 2, 32, 8)


@pytest.mark.parametrize("places", [(A, B, A, B), (A, None, A, None), (A, B, FAR, None),
                                    (A, B, None, FAR), (A, B, None, None), (A, None, B, None),
                                    (A, A, FAR, None), (A, A, None, None), (None,) * 4], ids=str)
def test_outputs_that_may_be(dsa, places):
    dsa._rotary_places(*places)


@pytest.mark.parametrize("places,match", [
    ((A, B, B, A), "apart from k"), ((A, B, None, A), "apart from q"),
    ((A, A, A, A), "apart from k"), ((A, A, None, A), "apart from q"),
    ((A, B, FAR, FAR), "q_out and k_out"), ((A, None, (1004, *A[1:]), None), "itself"),
    ((A, None, (9000, 8, 4, 2, 4, 64), None), "rows of q_out"),
], ids=str)
def test_outputs_that_may_not_be(dsa, places, match):
    with pytest.raises(ValueError, match=match):
        dsa._rotary_places(*places)


def test_another_default_device(dsa):
    """Rows are compared on the CPU wherever tensors are made by default."""
    with torch.device("meta"):
        assert dsa._rows_overlap((0, 8, 4, 2, 4, 64))
        assert not dsa._apart((0, 8, 4, 2, 24, 8), (4, 8, 4, 2, 24, 8))
