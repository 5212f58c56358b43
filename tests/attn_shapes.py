"""How the attention calls are cut (csrc/attn_prefill.hip, attn_paged.hip), for tests that
mean to reach one kernel: tile_shape, shares, streams and stream_row_tiles over again,
with the thresholds read from the sources. test_attn_shapes.py holds the rest of it
against gdn_attn_workspace_size, so a changed rule cannot move a test off its path
unnoticed."""

import os
import re
from types import SimpleNamespace

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "chunked_gated_delta_rule_amd", "csrc")


def _constants(*files):
    text = "".join(open(os.path.join(CSRC, f)).read() for f in files)
    return {n: int(v) for n, v in re.findall(r"^constexpr int (k\w+) = (\d+);", text, re.M)}


K = _constants("attn_prefill.hip", "attn_common.hpp")
ROWS, PAGES, SHARED = "rows", "pages", "shared"


def shape(c, keys, cus=256):
    group = c.h // c.hkv
    share = min(group, K["kMostShare"])
    while group % share:
        share -= 1
    room = c.max_pages * c.page_size
    longest = {SHARED: min(c.shared_max, room), PAGES: room}.get(keys, (c.tk_max or c.t_max) // c.n_max)

    def cut(rows):
        tt = rows // share
        return rows, tt, -(-c.t_max // tt) if keys == SHARED else c.t_max // tt + c.n_max

    rows, tt, slots = cut(K["kPartRows"])
    tiles = (slots if keys == SHARED else c.n_max * -(-(c.t_max // c.n_max) // tt)) * (c.h // share)
    n = cus // tiles if tiles else 1
    if n == 1 and (c.n_max == 1 or longest >= K["kTwoKeys"]):
        n = 2
    splits = min(max(min(n, longest // K["kSplitKeys"]), 1), K["kMostSplits"])
    if keys != SHARED and c.n_max > K["kMostTiled"]:
        splits = 1
    waves = 8
    if splits == 1 and keys != SHARED:
        waves = 8 if c.d == 256 or c.t_max // c.n_max >= K["kLongPrompt"] else 4
        rows, tt, slots = cut(32 * waves)
    parts = 0 if splits == 1 and keys != SHARED else slots * (c.h // share) * splits * rows
    return SimpleNamespace(waves=waves, rows=rows, share=share, tt=tt, slots=slots, splits=splits,
                           part_rows=parts)


def shares(c):
    return min(c.shared_max, c.max_pages * c.page_size) * c.n_max * c.hkv * c.d * 4 >= 256 << 20


def _rows_per_seq(c):
    return c.t_max * (c.h // c.hkv) // c.n_max


def streams(c):
    return _rows_per_seq(c) <= (64 if shares(c) else 32)


def stream_row_tiles(c):
    rt = 1
    while rt < (4 if c.d == 128 else 2) and _rows_per_seq(c) > 16 * rt:
        rt *= 2
    return rt


def workspace_size(c, cus=256):
    """gdn_attn_workspace_size from the shapes."""
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    tiles = lambda keys: up(shape(c, keys, cus).part_rows * c.d * 4) + \
        up(shape(c, keys, cus).part_rows * 8)  # noqa: E731
    if streams(c):
        rt = stream_row_tiles(c)
        slots = cus * (2 if rt * c.d <= 256 else 1) * 2 * 16 * rt
        done = c.t_max * c.h if shares(c) else 0
        paged = up(4) + up(c.t_max * c.h * 16) + up(slots * c.d * 4) + up(slots * 8) + \
            up(done * c.d * 4) + up(done * 8) + (tiles(SHARED) if shares(c) else 0)
    else:
        paged = tiles(PAGES)
    return max(tiles(ROWS), paged, 256)
