"""Sizes of the head that together reach each of its tiles: type, rows, vocabulary, width, and whether
the rows lie in strides that put them at any element.  None is a multiple of a tile or of a stage."""
SIZES = [
    ("f32", 2049, 32769, 772, False), ("f32", 506, 49821, 920, False), ("bf16", 400, 12001, 2056, False),
    ("f16", 400, 12001, 2056, False), ("bf16", 1103, 20011, 520, True), ("f16", 1103, 20011, 520, True),
    ("bf16", 1551, 10007, 1001, False), ("f16", 1551, 10007, 1001, False), ("bf16", 2, 306, 80, False),
    ("f32", 2, 370, 88, False), ("f16", 3, 315, 72, False), ("bf16", 8940, 2244, 168, False),
    ("f32", 2679, 5114, 272, True), ("bf16", 932, 20506, 284, True), ("f16", 1181, 20362, 274, False),
    ("f16", 10270, 1527, 472, True), ("bf16", 517, 50021, 1544, False), ("f16", 517, 50021, 1544, False),
    ("bf16", 2, 421, 77, False), ("f32", 2, 632, 88, True), ("f16", 3, 307, 170, False), ("f32", 42, 594, 72, False),
    ("f32", 564, 47120, 104, False),
]
