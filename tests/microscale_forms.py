"""Cases that reach every kernel form of the 4-bit products, among them workgroups
that run several tiles in turn, each with a ragged last stage (256 elements).  The
form that a case takes is asserted on the CPU (test_microscale_forms.py), the
results on the GPU (test_gpu_u_microscale_forms.py)."""

PAD = 7  # tasks behind the last expert's
FORMS = ("rows16", "rows32", "small", "mid", "wide", "big")

# (form, tiles in turn, counts, n, k, swiglu)
CASES = [
    ("rows16", False, [5, 0, 9, 7], 264, 4896, False),
    ("rows16", False, [5, 0, 9, 7], 264, 4896, True),
    ("rows32", False, [64, 65], 776, 4896, False),
    ("rows32", False, [33, 40], 904, 4896, True),
    # rows of less than 16 scales: a tile each
    ("small", False, [300, 3, 0, 70], 2056, 96, False),
    ("small", False, [200, 33], 1288, 384, True),
    ("small", False, [510, 3], 2056, 1120, False),
    ("small", False, [300, 0, 129], 1032, 736, True),
    ("small", True, [16 + e % 7 for e in range(60)], 1288, 800, False),
    ("small", True, [9 + e % 5 for e in range(60)], 650, 416, True),
    ("mid", False, [900, 600, 80], 2040, 864, False),
    ("mid", False, [1200, 700], 1016, 2080, True),
    ("mid", True, [4000, 40, 0, 3900], 2424, 448, False),
    ("mid", True, [4001, 0, 3899], 1210, 992, True),
    ("wide", False, [1020, 5], 4088, 5152, False),
    ("wide", False, [1020, 5], 2044, 5152, True),
    ("wide", True, [90 + e for e in range(34)], 2568, 2336, False),
    ("wide", True, [90 + e for e in range(34)], 1284, 2336, True),
    ("big", True, [5001, 0, 4900], 2312, 3360, False),
    ("big", True, [5001, 0, 4900], 1156, 3360, True),
]


def name(case):
    return "-".join(str(v) for v in case if not isinstance(v, list))
