"""Lengths that no row can have: who loses pages by them, and who does not."""
import numpy as np
import pytest
import torch

from test_pages_gpu import Both, ext, i32  # noqa: F401  (ext: the fixture)

pytestmark = pytest.mark.gpu
INT_MIN, INT_MAX = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("old,new", [((40, 33), (-1, 20)), ((40, 33), (INT_MIN, 33)), ((-1, 33), (0, 20)), ((40, 65), (3, 0)),
                                     ((40, INT_MAX), (40, 0)), ((INT_MIN, 33), (INT_MIN, 33)), ((40, 33), (65, 20))])
def test_release_leaves_rows_of_impossible_lengths_alone(ext, old, new):  # noqa: F811
    """Rows of 4 pages of 16: a length below 0 or above 64, old or new, keeps the row and its pages' counts;
    the other row is released as ever."""
    s = Both(ext, [40, 33], 16, 12, 4)
    ext.device_status()
    table, refs = s.table.cpu().numpy().copy(), s.refs.cpu().numpy().copy()
    for b in range(2):
        if all(0 <= x <= 64 for x in (old[b], new[b])):
            for i in range(-(-new[b] // 16), -(-old[b] // 16)):
                refs[table[b, i]] -= 1
                table[b, i] = -1
    ext.attn_sink_pages_release(s.table, s.refs, i32(old), i32(new), 16)
    assert ext.device_status() == ext._lib.DEV_SEQLEN_OOB
    np.testing.assert_array_equal(s.table.cpu().numpy(), table)
    np.testing.assert_array_equal(s.refs.cpu().numpy(), refs)


@pytest.mark.parametrize("bad", [-1, INT_MIN, 65, INT_MAX])
def test_compaction_takes_rows_of_impossible_lengths_along(ext, bad):  # noqa: F811
    """Their pages move like all that are counted, and their entries follow; entries that are none stay."""
    s = Both(ext, [40, 33, 64], 16, 40, 4, seed=3, kinds=("big",))
    ext.device_status()
    lens = s.lens.clone()
    lens[0] = bad
    before = s.table.cpu().numpy()
    want = s.m.compact()
    held = int(ext.attn_sink_pages_compact(s.caches, s.table, s.refs, lens, 16))
    assert ext.device_status() == ext._lib.DEV_SEQLEN_OOB
    assert held == want and np.any(before != s.m.table)
    s.same()


@pytest.mark.parametrize("bad", [-1, INT_MIN, 65, INT_MAX])
def test_fork_keeps_the_counts_of_what_it_cannot_tell(ext, bad):  # noqa: F811
    """A length below 0: a source without tokens, whose own pages stay counted.  One above the row: the
    whole row.  A source outside the table: a row without tokens.  No page that a row holds is free."""
    s = Both(ext, [40, 33, 64], 16, 40, 4, seed=4)
    ext.device_status()
    lens = s.lens.clone()
    lens[1] = bad
    old, refs = s.table.cpu().numpy(), s.refs.cpu().numpy()
    table, got = ext.attn_sink_pages_fork(s.table, s.refs, lens, i32([1, 0, 7, -2, 2]), 16)
    D = ext._lib
    assert ext.device_status() == D.DEV_SEQLEN_OOB | D.DEV_POOL | (0 if bad < 0 else D.DEV_PAGE_OOB)
    table, after = table.cpu().numpy(), s.refs.cpu().numpy()
    assert got.tolist() == [0 if bad < 0 else 64, 40, 0, 0, 64]
    rows = [[-1] * 4 if bad < 0 else old[1], old[0], [-1] * 4, [-1] * 4, old[2]]
    np.testing.assert_array_equal(table, rows)
    want = np.zeros_like(refs)
    np.add.at(want, table[table >= 0], 1)
    if bad < 0:
        want[old[1][old[1] >= 0]] += 1
    np.testing.assert_array_equal(after, want)
