"""What the page-management oracle reports of tables and counts that do not fit (CPU)."""
from oracle import manage


def _state():
    s = manage.State(40, 6, 6, 16)
    assert manage.reserve(s, [50, 33, 16, 0, 0, 0]) == set()
    s.lens = [50, 33, 16, 0, 0, 0]
    return s


def test_fork_of_a_last_page_beyond_the_pool():
    s = _state()
    s.table[1][2] = 40                        # the page that row 1 ends inside of
    assert manage.fork(s, [1, 0], [3, 4]) == {"bounds"}
    assert s.table[3] == s.table[1][:2] + [-1] * 4 and s.lens[3] == 33
    assert s.table[4][3] == 8 and s.lens[4] == 50 and s.ref[s.table[1][0]] == 2


def test_compact_with_entries_of_free_pages():
    for page in (5, 9):                       # below the pages in use, and above
        s = _state()
        s.ref[5] = 0                          # row 1 still names page 5
        s.table[2][1], s.ref[9] = 9, 1
        if page == 9:
            s.ref[9], s.ref[5] = 0, 1
        before = [row[:] for row in s.table]
        live, errors = manage.compact(s)
        assert errors == {"bounds"} and live == 8
        assert s.table[:2] == before[:2] and s.table[2][0] == 7
        assert s.table[2][1] == (5 if page == 5 else 9)
