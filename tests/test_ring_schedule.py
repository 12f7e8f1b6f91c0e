"""The host's account of the ring's tiles, and what the GPU tests built on it reach (no GPU)."""

import pytest

from tests import ring_schedule as rs


def test_by_hand():
    # 130 rows: 9 * 80, 5 * 96, 3 * 128, 2 * 192, 1 * 320; 517: 5 * 192 and 3 * 320 tie
    assert [rs.usual_height(m) for m in (1, 16, 17, 64, 130, 300, 517, 5000)] == [16, 16, 32, 64, 256, 128, 256, 256]
    # heights 16, 32 and 16; one tile of 64 columns costs least, and 64 columns run on 32 rows
    assert rs.tiles([3, 0, 17, 9], 256) == (64, {32: 3}, 24)
    # 16 rows only: no tile of 64 columns
    assert rs.tiles([3, 0, 16, 9], 256) == (128, {16: 3}, 24)
    # one expert of 618 rows, 216 columns: 3 tiles of 256 rows are 12 of 64 columns; cut to 32 rows (80 tiles)
    assert rs.tiles([618], 216) == (64, {32: 20}, 160)
    assert rs.tiles([256] * 64, 1024) == (256, {256: 64}, 256)
    assert rs.tiles([0, 0], 64)[1] == {}
    assert (rs.stages(256, 256, False), rs.stages(128, 256, True), rs.stages(64, 64, False)) == (2, 3, 6)
    assert (rs.slices(616, False), rs.slices(2400, True)) == (10, 10)


@pytest.mark.parametrize("mx", [False, True])
def test_every_tile_is_reached_with_its_ring_running_over(mx):
    assert len(rs.CONFIGS) == 14
    for height, width in rs.CONFIGS:
        sizes, cols = rs.launch_for(height, width)
        got, rows, G = rs.tiles(sizes, cols, height)
        assert (got, list(rows)) == (width, [height])
        assert sum(rows.values()) > G == rs.CUS, "several tiles a workgroup"
        s = rs.stages(height, width, mx)
        counts = [rs.slices(n, mx) for n in rs.lengths_for(height, width, mx)]
        assert {s - 1, s, s + 1, 10} == set(counts) and max(counts) >= s + 1
