"""Rows of nearly 2^31 tokens in the host's arithmetic (no GPU)."""
import pytest

import decode_attention_07_b200 as fd

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("L", [TOP, TOP - 1, TOP - 62, TOP - 63, TOP - 64, TOP - 255])
@pytest.mark.parametrize("splits", [1, 148, 1000])
def test_the_segments_of_a_row_cover_it(L, splits):
    d = fd.fd_segments(2, 1, TOP, [L, 5], splits)
    for row, n in ((0, L), (1, 5)):
        parts = sorted((int(b), int(e)) for r, b, e in zip(d["row"], d["begin"], d["end"]) if r == row)
        assert parts[0][0] == 0 and parts[-1][1] == n
        assert all(a[1] == b[0] and a[0] < a[1] for a, b in zip(parts, parts[1:]))


@pytest.mark.parametrize("L", [TOP, TOP - 62, TOP - 63])
def test_the_plan_of_a_long_row(L):
    assert fd.fd_plan_for_sms(1, 8, 1, 64, L, 148) == 148
    assert fd.fd_workspace_bytes(1, 8, 1, 64, L, 148) > 0
