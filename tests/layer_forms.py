"""Sizes of the 16-bit and 4-bit products by the form that they are meant to take
(few rows: rows of a tile / 16 and waves that share K;
many rows: tiles of 256 x 256), for the tests of the forms."""
from __future__ import annotations

# four, (rows of a tile / 16, waves that share K), counts of the groups, rows before and behind them, N, a short C and one
# of more stages than a turn of the loop has
STREAM = [
    (False, (1, 1), [1, 0, 16, 2, 17, 7, 3, 1] + [8] * 22 + [5, 0, 1], 1, 0, 523, 72, 1160),
    (False, (1, 2), [4] * 30 + [0, 1, 15], 0, 0, 262, 200, 1160),
    (False, (1, 4), [9, 7], 0, 0, 2050, 200, 1160),
    (False, (1, 8), [8], 0, 0, 33, 200, 2120),
    (False, (2, 1), [31, 32, 1] + [11] * 27 + [0, 2], 0, 0, 521, 136, 1096),
    (False, (2, 2), [16] * 29 + [33, 30, 1, 0], 0, 0, 259, 200, 1096),
    (False, (2, 4), [57], 0, 0, 2600, 72, 1096),
    (False, (2, 8), [8], 0, 0, 3909, 200, 2120),
    (False, (2, 8), [57], 0, 1, 780, 72, 2120),
    (False, (4, 1), [64, 65, 63, 128, 1, 40, 57, 62, 33], 0, 0, 1391, 72, 584),
    (False, (4, 2), [60, 64, 59, 63, 62], 0, 2, 1034, 72, 584),
    (False, (4, 2), [44], 0, 0, 7281, 136, 584),
    (False, (4, 4), [57], 0, 0, 1391, 200, 1096),
    (False, (8, 1), [80, 128, 40, 1, 70, 96, 0, 90, 7], 0, 0, 2050, 72, 328),
    (False, (8, 2), [58], 0, 0, 7281, 72, 584),
    (False, (8, 2), [100, 1, 70], 0, 0, 2602, 136, 584),
    (True, (1, 1), [1, 0, 16, 2, 17, 7, 3, 1] + [8] * 22 + [5, 0, 1], 1, 0, 523, 96, 2336),
    (True, (1, 2), [4] * 30 + [0, 1, 15], 0, 0, 262, 224, 4384),
    (True, (1, 4), [8], 0, 0, 33, 224, 8480),
    (True, (2, 1), [57], 0, 0, 7281, 96, 2336),
    (True, (2, 1), [32, 100, 39], 0, 0, 2601, 288, 2336),
    (True, (2, 2), [57], 0, 0, 778, 224, 4384),
    (True, (4, 1), [62], 0, 0, 1391, 224, 2336),
    (True, (4, 1), [64, 65, 57], 0, 0, 523, 96, 2336),
]

# every pair that the launches tell apart
STREAM_FORMS = {False: {(mt, share) for mt in (1, 2, 4, 8) for share in (1, 2, 4, 8) if share * mt <= 16},
                True: {(mt, share) for mt in (1, 2, 4) for share in (1, 2, 4) if share * mt <= 4}}

# four, counts, rows before and behind them, outputs (their width, whichever side of the weights it is), K: most groups
# end in a rest, of one row, 128 and just above
LARGE = [
    (False, [384, 130, 129, 513, 1], 0, 5, 10760, 64),
    (False, [128, 128, 256, 257, 255], 3, 0, 11000, 136),
    (True, [384, 130, 129, 513, 1], 0, 5, 5377, 160),
    (True, [128, 128, 256, 257, 255], 3, 0, 5600, 96),
]
