"""The kernel form that sizes choose for a 4-bit product (csrc/expert_forms.hpp,
compiled for the host): the cases that the GPU tests run reach every form and stay
with theirs, and every choice is one that the call accepts.  CPU only."""
import os
import shutil
import subprocess

import pytest

from tests import microscale_forms as F

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIM = os.path.join(ROOT, "tests", "host_sim")
CSRC = os.path.join(ROOT, "cartesian_routed_atomic_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang++ not installed")
    tmp = str(tmp_path_factory.mktemp("microscale_forms_sim"))
    exe = os.path.join(tmp, "microscale_forms_sim")
    r = subprocess.run([CLANG, "-std=c++20", "-O1", "-I", SIM, "-I", CSRC,
                        os.path.join(SIM, "microscale_forms_sim.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]

    def ask(cases):
        text = "".join(" ".join(str(int(v)) for v in c) + "\n" for c in cases)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert r.returncode == 0, r.stderr
        out = [[int(v) for v in line.split()] for line in r.stdout.splitlines()]
        assert len(out) == len(cases)
        return out
    yield ask
    shutil.rmtree(tmp, ignore_errors=True)


def test_cases_take_their_forms(choose):
    got = choose([(sum(c) + F.PAD, len(c), n, k, sw) for _, _, c, n, k, sw in F.CASES])
    wrong = [(F.name(c), F.FORMS[f], tiles, blocks) for c, (f, tiles, blocks) in zip(F.CASES, got)
             if F.FORMS[f] != c[0] or (blocks < tiles) != c[1]]
    assert not wrong
    for form in F.FORMS:
        for sw in (False, True):
            assert any(c[0] == form and c[5] == sw for c in F.CASES)


def test_short_rows_have_a_workgroup_for_every_tile(choose):
    for k in (32, 128, 256, 384):
        (_, tiles, blocks), = choose([(60000, 1, 4096, k, 0)])
        assert tiles == blocks
    (_, tiles, blocks), = choose([(60000, 1, 4096, 416, 0)])
    assert blocks in (256, 512) and tiles > blocks
