"""The tiles that the data gradient and the 4-bit product choose, worked out on the host.

Written from the rules that ``gg_ring.h`` states (heights by the forward product's
choice, cut where the launch leaves CUs idle; one width by the cost of its rounds),
so that tests can say which tiles a case runs on. ``CUS`` is the MI355X's.
"""

CUS = 256
HEIGHTS = (16, 32, 64, 128, 256)
WIDTHS = (256, 128, 64)
RING_BYTES = 155 * 1024


def _up(a, b):
    return -(-a // b)


def stages(height, width, mx):
    """LDS stages of a tile: a slice is 128 bytes a row, with 8 scale bytes in 4 bits."""
    return min(6, RING_BYTES // ((height + width) * (136 if mx else 128)))


def slices(length, mx):
    """Slices of a sum over ``length`` values of 2 bytes, or of 4 bits."""
    return _up(length, 256 if mx else 64)


def usual_height(rows):
    """Smallest ceil(rows / h) * (h + 64), the taller at a tie."""
    return min(HEIGHTS, key=lambda h: (_up(rows, h) * (h + 64), -h))


def workgroups(M_cap, E, cols, bm):
    bound = (M_cap // (bm or 16) + E) * _up(cols, 64)
    return _up(min(bound, CUS), 8) * 8


def tiles(sizes, cols, bm=0, M_cap=None):
    """(width, {tile height: its row tiles}, workgroups) of a launch; heights as the tiles run."""
    sizes = [int(m) for m in sizes]
    G = workgroups(sum(sizes) if M_cap is None else M_cap, len(sizes), cols, bm)
    heights = [bm or usual_height(m) for m in sizes if m > 0]
    rows = [m for m in sizes if m > 0]
    if not rows:
        return None, {}, G
    tallest = max(heights)

    def row_tiles():
        return sum(_up(m, min(h, tallest)) for m, h in zip(rows, heights))

    narrow = row_tiles() * _up(cols, 64)
    if bm == 0 and tallest > 32 and 2 * narrow <= G:
        n = 2 * narrow
        while tallest > 32 and n <= G:
            tallest //= 2
            n *= 2
    total = row_tiles()
    # 64 columns need 32 rows
    able = [w for w in WIDTHS if w >= 128 or tallest > 16]
    width = min(able, key=lambda w: (_up(total * _up(cols, w), G) * (tallest + w + 96), -w))
    out = {}
    for m, h in zip(rows, heights):
        h = min(h, tallest)
        run = max(h, 32) if width == 64 else h
        out[run] = out.get(run, 0) + _up(m, h)
    return width, out, G


# The configurations there are, and a launch that runs on each: a ragged last row tile
# for most experts, an empty and a one-row expert, ragged columns, more tiles than
# workgroups (so that a tile's first slices load while the one before it is stored).
CONFIGS = [(h, w) for h in HEIGHTS for w in WIDTHS if (h, w) != (16, 64)]


def launch_for(height, width):
    """(sizes, columns); the tile height is given with the call."""
    per = 47 if height == 16 else 27
    sizes = [per * height - (7 * i) % height for i in range(9)]
    return sizes[:3] + [0] + sizes[3:] + [1, height + 1] + [per * height], {64: 56, 128: 120, 256: 248}[width]


def lengths_for(height, width, mx):
    """Lengths of the sum: S - 1, S, S + 1 and 10 slices, the last of which is not full."""
    s = stages(height, width, mx)
    unit, tail = (256, 96) if mx else (64, 40)
    return [unit * (k - 1) + tail for k in sorted({s - 1, s, s + 1, 10})]
