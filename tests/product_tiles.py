"""Sizes at which the experts' products change their tile, by the rule as it
stands: (expected_rows, (token rows, output channels, weights read once)).
Each list is one set of sizes, run over all of its expected_rows; both sides of
every change that the sizes reach are there."""

# 16 experts, inter_features 1152: all five gated tiles.
GATED = dict(experts=16, out=1152, rows=1600, cases=[
    (1, (32, 128, True)), (320, (32, 128, True)), (335, (32, 128, True)),
    (336, (32, 128, False)), (671, (32, 128, False)),
    (672, (64, 128, True)), (704, (64, 128, True)), (719, (64, 128, True)),
    (720, (64, 128, False)), (1536, (64, 128, False)), (1551, (64, 128, False)),
    (1552, (128, 128, False)), (1600, (128, 128, False)),
])
# 2 experts, 7456 channels: all plain tiles but the one for few rows of many experts.
PLAIN_FEW = dict(experts=2, out=7456, rows=1101, cases=[
    (1, (32, 128, True)), (33, (32, 128, True)),
    (34, (32, 128, False)), (255, (32, 128, False)),
    (256, (64, 256, False)), (511, (64, 256, False)),
    (512, (128, 256, False)), (1023, (128, 256, False)),
    (1024, (256, 256, False)), (1101, (256, 256, False)),
])
# 16 experts, 4224 channels: that one, and its neighbours.
PLAIN_MANY = dict(experts=16, out=4224, rows=900, cases=[
    (256, (32, 128, True)), (271, (32, 128, True)),
    (272, (64, 256, True)), (783, (64, 256, True)),
    (784, (128, 256, False)), (900, (128, 256, False)),
])
# One dense product of 4224 channels.
DENSE = dict(experts=1, out=4224, rows=1100, cases=[
    (16, (32, 128, True)), (17, (32, 128, False)), (495, (32, 128, False)),
    (496, (64, 256, False)), (991, (64, 256, False)),
    (992, (128, 256, False)), (1100, (128, 256, False)),
])

GATED_TILES = {(32, 128, True), (32, 128, False), (64, 128, True), (64, 128, False),
               (128, 128, False)}
PLAIN_TILES = {(32, 128, True), (32, 128, False), (64, 256, True), (64, 256, False),
               (128, 256, False), (256, 256, False)}
