"""The page tables' oracle by hand."""
from oracle import pages as op


def test_lowest_free_pages_in_order_of_sequence_and_entry():
    table, refs = [[4, -1, -1], [-1, 9, -1]], [0, 1, 0, 0, 1, 0]
    missing, slots, positions = op.reserve(table, refs, [3, 0], [6, 9], 4)
    assert table == [[4, 0, 2], [3, 5, -1]] and refs == [1, 1, 1, 1, 1, 1] and missing == [0, 1]
    assert slots == [19, 0, 1, 2, 3, 8, 12, 13, 14, 15, 20, 21, 22, 23, -1]
    assert positions == [3, 4, 5, 6, 7, 8] + list(range(9))


def test_release_and_shared_pages():
    table, refs = [[0, 1, 2], [0, 3, -1]], [2, 1, 1, 1]
    op.release(table, refs, [5, 0], 4)
    assert table == [[0, 1, -1], [-1, -1, -1]] and refs == [1, 1, 0, 0]
    op.release(table, refs, [0, 0], 4)
    assert refs == [0, 0, 0, 0]


def test_depths_are_positions_and_tables_end():
    table, refs = [[-1]], [0, 0]
    missing, slots, positions = op.reserve(table, refs, [2], [4], 4, depth=[0, 1, 1, 2])
    assert missing == [0] and slots == [2, 3, -1, -1] and positions == [2, 3, 3, 4]
