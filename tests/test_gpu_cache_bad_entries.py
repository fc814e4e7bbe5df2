"""Lists and tables that contradict themselves: a fork of a row that the same
list makes, an entry that holds a page without references."""
import pytest

from _pool import REFS, ROW, Pool
from test_gpu_cache import Device, _cuda  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("parents,children", [([0, 4], [4, 5]), ([4, 0], [5, 4]), ([6], [6]),
                                              ([0, 4, 5], [4, 5, 6])])
def test_fork_of_a_row_that_the_list_makes(parents, children):
    """Parents are read as they were: the child of such a row would be empty."""
    p = Pool(20, 8, 4, 4, [16])
    p.fill_row(0, 6)
    d = Device(p)
    for q in (p, d):
        q.fork(parents, children)
    assert p.lens[[5, 6]].tolist() == [0, 0]  # the plain model makes them empty rows
    p.err |= ROW
    d.check(p)


def test_fork_of_unused_rows_alone():
    """An unused row is a parent like any other: its child stays unused."""
    p = Pool(20, 8, 4, 4, [16])
    p.fill_row(0, 6)
    p.fill_row(1, 3)
    d = Device(p)
    for q in (p, d):
        q.fork([2, 0, 2], [4, 5, 6])
        q.fork([1], [3])
    assert p.err == 0
    d.check(p)


def test_fork_of_a_used_row_that_the_list_names_as_a_child():
    """That child is refused, so the parent is what it was."""
    p = Pool(20, 8, 4, 4, [16])
    p.fill_row(0, 6)
    p.fill_row(1, 9)
    d = Device(p)
    for q in (p, d):
        q.fork([0, 1], [1, 2])
    assert p.err == ROW and p.lens[:3].tolist() == [6, 9, 9]
    d.check(p)

def test_compact_leaves_no_entry_on_a_page_that_another_row_gets():
    """An entry below the border whose page nobody counts: the page is a hole, and
    another row's page moves there."""
    p = Pool(12, 3, 4, 4, [16, 8])
    p.fill_row(0, 11, [5, 0, 9])
    p.fill_row(1, 7, [2, 7])
    p.refs[2] = 0
    d = Device(p, extra_cols=1)
    assert d.compact() == p.compact() == 4
    assert p.table[0, :3].tolist() == [1, 0, 3] and p.table[1, :2].tolist() == [2, 2]
    p.table[1, 0] = -1
    p.err |= REFS
    d.check(p)
