"""The kernel form that sizes and types choose (csrc/expert_forms.hpp, compiled
for the host): the cases that the GPU tests run reach every form, and stay with
theirs when a rule changes.  CPU only."""
import os
import shutil
import subprocess

import pytest

from tests import expert_forms as F
from tests import test_gpu_k_experts as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIM = os.path.join(ROOT, "tests", "host_sim")
CSRC = os.path.join(ROOT, "cartesian_routed_atomic_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang++ not installed")
    tmp = str(tmp_path_factory.mktemp("expert_forms_sim"))
    exe = os.path.join(tmp, "expert_forms_sim")
    r = subprocess.run([CLANG, "-std=c++20", "-O1", "-I", SIM, "-I", CSRC,
                        os.path.join(SIM, "expert_forms_sim.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]

    def ask(lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True,
                           timeout=60)
        assert r.returncode == 0, r.stderr
        out = [[int(v) for v in line.split()] for line in r.stdout.splitlines()]
        assert len(out) == len(lines)
        return out
    yield ask
    shutil.rmtree(tmp, ignore_errors=True)


def product(dt, M, E, n, k, transpose=False, swiglu=False):
    return f"p {F.TYPES[dt]} {M} {E} {n} {k} {int(transpose)} {int(swiglu)}"


def test_product_cases_take_their_forms(choose):
    got = choose([product(dt, sum(c) + F.PAD, len(c), n, k, tr, sw)
                  for _, dt, c, n, k, tr, sw in F.PRODUCTS])
    wrong = [(F.name(c), F.FORMS[g]) for c, (g,) in zip(F.PRODUCTS, got) if F.FORMS[g] != c[0]]
    assert not wrong
    # every form that is compiled, in each of its types and modes
    reached = {(c[0], c[1], c[5], c[6]) for c in F.PRODUCTS}
    for dt in ("bf16", "i8"):
        for form in ("rows16", "rows32", "rows64", "small", "mid", "wide", "big"):
            assert {(form, dt, False, False), (form, dt, False, True)} <= reached
            assert dt == "i8" or form.startswith("rows") or (form, dt, True, False) in reached
    for form in ("rows16", "rows32", "rows64", "f32"):
        assert {(form, "f32", False, False), (form, "f32", False, True)} <= reached
    assert ("f32", "f32", True, False) in reached


def test_weight_gradient_cases_take_their_tiles(choose):
    got = choose([f"w {int(dt == 'bf16')} {sum(c) + F.PAD} {len(c)} {n} {k}"
                  for _, _, dt, c, n, k in F.WEIGHT_GRADIENTS])
    for case, (tile, part, slots) in zip(F.WEIGHT_GRADIENTS, got):
        assert (tile, part > 0) == case[:2], case
        # an expert in several parts, where there are parts
        assert part == 0 or max(case[3]) > part and slots >= 2, case
    assert {c[:3] for c in F.WEIGHT_GRADIENTS} == {
        (64, False, "f32"), (64, True, "f32"), *((t, p, "bf16") for t in (64, 128, 256)
                                                 for p in (False, True))}


def test_steady_loops_are_reached():
    """Eight stages or more in every case."""
    for form, dt, _, n, k, tr, _ in F.PRODUCTS:
        size = {"bf16": 2, "i8": 1, "f32": 4}[dt]
        stages = -(-(n if tr else k) * size // 64)
        assert stages >= (64 if form.startswith("rows") else 11), (form, dt)
        assert (n if tr else k) * size % 64, (form, dt)
    for _, _, dt, counts, _, _ in F.WEIGHT_GRADIENTS:
        assert max(counts) >= 8 * (32 if dt == "bf16" else 16)


def test_forms_of_the_other_gpu_tests(choose):
    """What the cases of test_gpu_k_experts.py run: those that are named for a form,
    but for "mid", which takes 128 x 256 tiles (128 x 128 ones run above)."""
    for n, form in (("rows_32", "rows32"), ("rows_64", "rows64"), ("small", "small"),
                    ("mid", "wide"), ("wide", "wide"), ("big", "big"), ("big_last_rows", "big")):
        counts, width, k = K.WIDE[n]
        (got,), = choose([product("bf16", sum(counts) + K.PAD, len(counts), width, k)])
        assert F.FORMS[got] == form, n
    # the float32 sums in blocks: the forward case there takes the rows kernel
    (got,), = choose([product("f32", 610, 4, 200, 3424)])
    assert F.FORMS[got] == "rows64"
    # and the one beside it in test_gpu_p_expert_forms.py the tiles
    for steps in (1000, 3424):
        (got,), = choose([product("f32", 610, 4, 840, steps)])
        assert F.FORMS[got] == "f32"
        (tile, part, _), = choose([f"w 1 {steps} 1 8192 8192"])
        assert (tile, part) == (256, 0)
