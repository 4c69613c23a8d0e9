"""The tile search of the expert operators (csrc/expert_tiles.hpp), compiled for
the host and run on the wave model of tests/host_sim/ with the address and
undefined-behaviour sanitizers (an index that passes 32 bits stops the run).
CPU only.

Whatever the offsets hold, a workgroup's tile lies within the tasks; with
offsets in order the tiles cover every task and column once."""
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIM = os.path.join(ROOT, "tests", "host_sim")
CSRC = os.path.join(ROOT, "cartesian_routed_atomic_amd", "csrc")
CLANG = "/opt/rocm/llvm/bin/clang++"
TILES, PARTS, BY_SIZE = range(3)


@pytest.fixture(scope="module")
def sim(tmp_path_factory):
    if not os.path.exists(CLANG):
        pytest.skip("ROCm clang++ not installed")
    tmp = str(tmp_path_factory.mktemp("expert_tiles_sim"))
    exe = os.path.join(tmp, "expert_tiles_sim")
    r = subprocess.run([CLANG, "-std=c++20", "-O1", "-g", "-fno-sanitize-recover=all",
                        "-fsanitize=address,undefined", "-I", SIM, "-I", CSRC,
                        os.path.join(SIM, "expert_tiles_sim.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    yield exe, tmp
    shutil.rmtree(tmp, ignore_errors=True)


def run(sim, mode, off, M, bm, n_nt, ids, slots=0, blocks=0):
    exe, tmp = sim
    fin, fout = os.path.join(tmp, "in.bin"), os.path.join(tmp, "out.bin")
    with open(fin, "wb") as f:
        np.array([mode, len(off) - 1, M, bm, n_nt, slots, blocks, len(ids)], np.int32).tofile(f)
        np.asarray(ids, np.int32).tofile(f)
        np.asarray(off, np.int32).tofile(f)
    r = subprocess.run([exe, fin, fout], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0, r.stderr[-3000:]
    return np.fromfile(fout, np.int32).reshape(-1, 5)


def launched(M, E, bm, n_nt):
    """Workgroups of a launch: row tiles that E experts of M tasks can have."""
    return (M + min(E, M) * (bm - 1)) // bm * n_nt


def in_order(counts):
    return np.concatenate([[0], np.cumsum(counts)])


@pytest.mark.parametrize("E,bm,n_nt,tail", [(1, 64, 3, 0), (5, 16, 1, 9), (64, 32, 7, 0),
                                            (65, 64, 13, 3), (300, 16, 2, 40)])
def test_tiles_cover_every_task_once(sim, E, bm, n_nt, tail):
    rng = np.random.default_rng(E)
    counts = rng.integers(0, 3 * bm, E) * (rng.random(E) < 0.7)
    off = in_order(counts)
    M = int(off[-1]) + tail
    nb = launched(M, E, bm, n_nt)
    out = run(sim, TILES, off, M, bm, n_nt, range(nb))
    seen = np.zeros((M, n_nt), int)
    for e, m0, m1, nt, _ in out:
        if m0 >= m1:
            continue
        assert off[e] <= m0 < m1 <= off[e + 1] and m1 - m0 <= bm and (m0 - off[e]) % bm == 0
        seen[m0:m1, nt] += 1
    assert (seen[:off[-1]] == 1).all() and (seen[off[-1]:] == 0).all()


def test_dense_tiles_cover_every_task_once(sim):
    M, bm, n_nt = 700, 128, 9
    nb = launched(M, 1, bm, n_nt)
    seen = np.zeros((M, n_nt), int)
    exe, tmp = sim
    for e, m0, m1, nt, _ in run(sim, TILES, [0, M], M, bm, n_nt, range(nb), blocks=nb):
        assert e == 0 and m1 - m0 <= bm
        seen[m0:m1, nt] += 1
    assert (seen == 1).all()


@pytest.mark.parametrize("E,part,tiles", [(3, 512, 2), (70, 1024, 1), (200, 512, 3)])
def test_parts_cover_every_task_once_and_slots_do_not_meet(sim, E, part, tiles):
    rng = np.random.default_rng(E)
    off = in_order(rng.integers(0, 4 * part, E) * (rng.random(E) < 0.8))
    M = int(off[-1])
    slots = min(M // part + E, 2 * M // part)
    nb = launched(M, E, part, tiles)
    out = run(sim, PARTS, off, M, part, tiles, range(nb), slots)
    seen, used = np.zeros((M, tiles), int), set()
    for e, lo, hi, slot, tile in out:
        if lo >= hi:
            continue
        assert off[e] <= lo < hi <= off[e + 1]
        seen[lo:hi, tile] += 1
        assert (slot >= 0) == (off[e + 1] - off[e] > part) and slot < slots
        assert (slot, tile) not in used or slot < 0
        used.add((slot, tile))
    assert (seen == 1).all()


# Offsets that go back and forth: every second expert has all M tasks, so the
# tiles that the experts ask for pass 2^31 and 2^32 in sum, within one lane
# (E / 128 experts of it) or over the lanes, although a launch stays below 2^24.
BACK_AND_FORTH = [
    # E, M, bm, n_nt
    (1 << 12, 1 << 26, 16, 1),        # 2^33 over the lanes
    (1 << 16, 1 << 26, 16, 1),        # 2^31 in every lane
    (3 << 15, 1 << 26, 16, 1),        # 3 x 2^30 in every lane
    (1 << 17, 1 << 26, 16, 1),        # 2^32 in every lane
    (3000, 1 << 22, 64, 130),         # row tiles fit, times columns they do not
    (6, 1 << 26, 16, 1),
]


@pytest.mark.parametrize("E,M,bm,n_nt", BACK_AND_FORTH)
@pytest.mark.parametrize("low", [0, 7])
def test_tiles_of_overlapping_offsets_stay_within_the_tasks(sim, E, M, bm, n_nt, low):
    off = np.where(np.arange(E + 1) % 2, M - low, low)
    off[::5] = low                                    # not the same in every lane
    nb = launched(M, E, bm, n_nt)
    assert nb < 1 << 24
    rng = np.random.default_rng(E)
    ids = np.unique(np.concatenate([[0, 1, nb - 1, nb // 2], rng.integers(0, nb, 12)]))
    for e, m0, m1, nt, _ in run(sim, TILES, off, M, bm, n_nt, ids):
        assert 0 <= e < E and 0 <= m0 <= m1 <= M and 0 <= nt < n_nt


@pytest.mark.parametrize("E,M,part,tiles", [(4000, 1 << 30, 512, 2), (700, 1 << 30, 1024, 5)])
def test_parts_of_overlapping_offsets_stay_within_the_tasks(sim, E, M, part, tiles):
    off = np.where(np.arange(E + 1) % 2, M, 0)
    slots = min(M // part + E, 2 * M // part)
    nb = launched(M, E, part, tiles)
    rng = np.random.default_rng(E)
    ids = np.unique(np.concatenate([[0, nb - 1], rng.integers(0, nb, 12)]))
    for e, lo, hi, slot, tile in run(sim, PARTS, off, M, part, tiles, ids, slots):
        assert 0 <= e < E and 0 <= lo <= hi <= M and -1 <= slot < slots and 0 <= tile < tiles
        # a partial sum's place is never taken for dW's
        assert lo == hi or (slot >= 0) == (hi - lo < M or M <= part)


def test_experts_by_size(sim):
    rng = np.random.default_rng(3)
    E = 150
    counts = rng.integers(0, 40, E) * (rng.random(E) < 0.6)
    off = in_order(counts)
    out = run(sim, BY_SIZE, off, int(off[-1]), 0, 0, range(E))
    want = np.concatenate([first + np.argsort(-counts[first:first + 64], kind="stable")
                           for first in range(0, E, 64)])
    np.testing.assert_array_equal(out[:, 0], want)
    np.testing.assert_array_equal(out[:, 1], off[want])
    np.testing.assert_array_equal(out[:, 2], off[want + 1])
