"""CPU tests of the paged cache's oracle (oracle/paged.py) against cases worked by hand."""
import numpy as np

from oracle import paged as op


def _i32(*v):
    return np.array(v, dtype=np.int32)


def test_pages_given_back_are_taken_first_in_order():
    table = np.array([[5, 6, 7], [1, -1, -1], [-1, -1, -1]], dtype=np.int32)
    free = _i32(9, 8, 3, 0, 0, 0, 0, 0, 0, 0)
    # request 0 gives pages 6 and 7 (6 uppermost), request 1 misses one, request 2 two
    t, h, f, n, s, e = op.page_assign(table, _i32(3, 1, 0), free, 3, _i32(4, 8, 5), 4, _i32(0, 2, 3), 3)
    assert t.tolist() == [[5, 6, 7], [1, 6, -1], [7, 3, -1]] and h.tolist() == [1, 2, 2]
    assert n == 2 and f[:2].tolist() == [9, 8] and e == 0
    assert s.tolist() == [[20, 21, 22], [6, 7, 24], [31, 12, -1]]


def test_growing_and_shrinking_back_restores_the_state():
    rng = np.random.RandomState(1)
    table = np.full((5, 6), -1, dtype=np.int32)
    ids = rng.permutation(30).astype(np.int32)
    held = _i32(0, 2, 1, 3, 0)
    for b in range(5):
        table[b, :held[b]] = ids[held[:b].sum():held[:b + 1].sum()]
    free = np.concatenate([ids[6:], ids[:6]])
    old = (held * 8).astype(np.int32)
    t, h, f, n, _, e = op.page_assign(table, held, free, 24, old + 20, 8)
    assert e == 0 and n == 24 - 15
    t, h, f, n, _, e = op.page_assign(t, h, f, n, old, 8)
    assert n == 24 and (f == free).all() and (h == held).all()


def test_shortage_refuses_from_the_first_that_is_not_covered():
    table = np.full((4, 3), -1, dtype=np.int32)
    free = _i32(0, 1, 2)
    t, h, f, n, s, e = op.page_assign(table, _i32(0, 0, 0, 0), free, 3, _i32(8, 8, 4, 0), 4, _i32(0, 0, 0, 0), 1)
    assert h.tolist() == [2, 0, 0, 0] and n == 1 and e == 2 and s[:, 0].tolist() == [8, -1, -1, -1]
    t, h, f, n, s, e = op.page_assign(table, _i32(0, 4, 0, 0), free, 3, _i32(4, 4, 13, -1), 4)
    assert h.tolist() == [1, 4, 0, 0] and e == 2


def test_filters_by_hand():
    l = np.log(np.array([0.1, 0.4, 0.1, 0.4]))
    assert op.sample(l, 0.0, 1.0, 0, 1.0, 0.0)[0] == 0
    assert op.sample(l, 0.95, 1.0, 0, 1.0, 0.0)[0] == 3
    assert op.sample(l, 0.0, 1.0, 1, 1.0, 0.0)[0] == 1            # equal logits: the lower index is first
    assert op.sample(l, 0.9, 1.0, 0, 0.5, 0.0)[0] == 3            # 0.4 < 0.5: both of the largest
    assert op.sample(l, 0.0, 1.0, 0, 0.85, 0.0)[0] == 0           # and the first of the next
    assert op.sample(l, 0.99, 1.0, 0, 1.0, 0.5)[0] == 3 and op.sample(l, 0.0, 1.0, 0, 1.0, 0.5)[0] == 1
    assert op.sample(l, 0.7, 0.0, 0, 1.0, 0.0)[0] == 1
    assert abs(op.sample(l, 0.0, 1.0, 1, 1.0, 0.0)[1] - math_log(0.4)) < 1e-12


def math_log(x):
    import math
    return math.log(x)
