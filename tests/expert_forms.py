"""Cases that reach every kernel form of the expert operators, each with a
contraction long enough for the pipeline's steady loop (eight stages of 64 bytes
of the contraction; 32 bf16, 64 int8, 16 float32) and a ragged last stage.  The
form that a case takes is asserted on the CPU (test_expert_forms.py), the results
on the GPU (test_gpu_p_expert_forms.py)."""

PAD = 7  # tasks behind the last expert's
TYPES = {"f32": 0, "bf16": 1, "i8": 2}
FORMS = ("rows16", "rows32", "rows64", "f32", "small", "mid", "wide", "big")

# form: counts, output columns of W (with swiglu both halves)
PRODUCT_SHAPES = {
    "rows16": ([5, 0, 9, 16], 264),
    "rows32": ([64, 65], 520),
    "rows64": ([129, 200], 264),
    "small": ([510, 3], 2056),
    "mid": ([600, 500], 2040),
    "wide": ([1020, 5], 4088),
    "big": ([2041, 1800], 3848),
    "f32": ([150, 170, 90, 200], 1032),
}
# the rows kernels give each of eight waves an eighth of the stages: more than
# twice the four that a wave has in flight
LENGTHS = {"rows": {"bf16": 2408, "i8": 4816, "f32": 1204},
           "tile": {"bf16": 32 * 10 + 8, "i8": 64 * 10 + 16, "f32": 16 * 21 + 4}}


def _products():
    """(form, type, counts, n, k, transpose, swiglu)"""
    for form, (counts, width) in PRODUCT_SHAPES.items():
        for dt in TYPES:
            rows = form.startswith("rows")
            if not rows and (form == "f32") != (dt == "f32"):
                continue
            length = LENGTHS["rows" if rows else "tile"][dt]
            yield form, dt, counts, width, length, False, False
            yield form, dt, counts, width // 2, length, False, True
            if not rows and dt != "i8":
                yield form, dt, counts, length, width, True, False


PRODUCTS = list(_products())

# (tile, in parts, type, counts, n, k)
WEIGHT_GRADIENTS = [
    (64, False, "bf16", [300, 0, 333, 280], 136, 200),
    (64, True, "bf16", [3001, 40, 0, 700], 72, 136),
    (64, False, "f32", [300, 0, 333, 280], 136, 200),
    (64, True, "f32", [3001, 40, 0, 700], 72, 136),
    (128, False, "bf16", [300, 290, 310, 301, 257], 1032, 1016),
    (128, True, "bf16", [5001], 1016, 1032),
    (128, True, "bf16", [2500, 9, 1100], 1160, 1032),
    (256, False, "bf16", [300 + 3 * e for e in range(13)], 1032, 760),
    (256, True, "bf16", [8001], 2040, 2056),             # room for the short part in a round
    (256, True, "bf16", [3300, 0, 500, 200, 150, 33], 2040, 2056),  # and none
]


def name(case):
    return "-".join(str(v) for v in case if not isinstance(v, list))
