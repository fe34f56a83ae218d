"""State-space operators without a GPU: the splits that the cases of test_state_space_edges_gpu.py are made for."""

import pytest

from test_state_space_edges_gpu import ROWS, WIDE, norm_groups, scan_splits


@pytest.mark.parametrize("case", WIDE, ids=["x".join(map(str, c[:5])) for c in WIDE])
def test_scan_cases_have_their_splits(case):
    *sizes, wide, segments, _ = case
    assert scan_splits(*sizes) == [(wide, segments)]


@pytest.mark.parametrize("D, rows", ROWS)
def test_norm_cases_have_three_rows_a_workgroup(D, rows):
    groups = -(-rows // 3)
    assert rows % 3 and groups <= norm_groups(rows, D) < groups + 256 / (12 * D)


@pytest.mark.parametrize("D", [1, 40, 512, 1024, 2048, 2560, 4096, 8192])
def test_norm_workgroups_have_at_most_128_rows(D):
    for rows in (1, 127, 128, 129, 4096, 32768, 32769, 393216, 393217, 1 << 20, (1 << 24) + 1):
        groups = norm_groups(rows, D)
        assert 1 <= groups and rows <= 128 * (groups + 256 / (12 * D))
