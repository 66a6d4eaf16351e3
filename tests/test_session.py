"""Host logic of the session classes, without a GPU."""
import numpy as np
import pytest

from kv_cache_serving_gb300 import session


def test_page_rows():
    """Rows that each page holds: of the requests that map it, the most; entries of -1 (evicted
    pages) and past a request's last row count for nothing."""
    table = np.array([[4, 0, 2], [4, 3, -1], [-1, 5, 6], [1, 1, 1]])
    rows = session.page_rows(table, [40, 17, 18, 0], 8)
    assert rows.tolist() == [16, 0, 8, 1, 16, 2, 0, 0]
    assert session.page_rows(table[::-1], [0, 18, 17, 40], 8).tolist() == rows.tolist()
    assert session.page_rows(np.zeros((0, 3), int), [], 2).tolist() == [0, 0]


def test_page_rows_refuses_lengths_past_the_table():
    with pytest.raises(ValueError):
        session.page_rows(np.zeros((1, 2), int), [33], 4)
    with pytest.raises(ValueError):
        session.page_rows(np.full((1, 2), 4), [20], 4)
