"""Which tile kernel the 8-bit product takes, by the rules of spec_logits.hip, whose numbers are read from the source;
and the shapes that the tests run, one at least for each kernel."""
import os
import re

from speculative_sampling_verification_verify_amd import build

_SRC = open(build.LOGITS_SRC).read()
(_TABLE,) = re.findall(r"tile\[\] = \{(.*)\};", _SRC)
TILES = [tuple(map(int, t)) for t in re.findall(r"\{(\d+), (\d+), (\d+)\}", _TABLE)]          # cn, mt, us
((WIDE4, WIDE),) = [tuple(map(int, t)) for t in re.findall(r"\(mt >= 4 \? (\d+) : (\d+)\)", _SRC)]
(EXACT_ROWS,) = map(int, re.findall(r"F8_EXACT_ROWS = (\d+);", _SRC))
assert len(TILES) == 4

up = lambda a, b: -(-a // b)


def form(R, N, f8):
    """(cn, mt, f8) of a call of more than 16 rows."""
    if f8 and R > EXACT_ROWS:
        mt = min(range(5, 0, -1), key=lambda m: up(R, 64 * m) * m)     # the widest of the least padded
        rows = up(R, 64 * mt)
        wide = up(up(N, 256) * rows, 256) * 100 <= up(up(N, 128) * rows, 256) * (WIDE4 if mt >= 4 else WIDE)
        return (2 if wide else 1), mt, True
    cn, mt, _ = min(TILES, key=lambda t: up(up(N, 128 * t[0]) * up(R, 64 * t[1]), 256) * t[2])
    return cn, mt, False


def row_blocks(R, f8):
    """Blocks of 32 rows of the workspace."""
    if f8 and R > EXACT_ROWS:
        mt = form(R, 1, True)[1]
        return up(R, 64 * mt) * 2 * mt
    return up(R, 128) * 4


# (R, K, N, 8-bit products): more blocks of K than a workgroup's buffers (at most six) and a last one that is short,
# rows and columns that end inside a tile, one and several row tiles.
SHAPES = [
    (40, 1040, 300, False), (40, 1040, 32897, False), (100, 912, 17001, False), (100, 1040, 33001, False), (450, 912, 20001, False),
    (260, 1040, 17001, False), (400, 1040, 300, True), (400, 1040, 5001, True), (100, 1040, 400, True), (100, 1040, 32897, True),
    (130, 1040, 400, True), (130, 1040, 32897, True), (200, 1040, 400, True), (200, 1040, 32897, True), (300, 1040, 400, True),
    (300, 1040, 32897, True), (500, 912, 25001, True), (640, 1040, 26001, True)]
# The longest K: the weights' scales fill their place in LDS.
LONG = [(4100, 1101, False), (40, 32897, False), (4097, 4500, True)]
