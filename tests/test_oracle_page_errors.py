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
