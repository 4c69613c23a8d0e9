"""The limits of the expert operators, on both sides: host checks that return
before any HIP call, so they need no GPU.  Where a size is taken, a later check
(no tasks, no workspace) ends the call."""
import ctypes

import pytest

B = pytest.importorskip("cartesian_routed_atomic_amd.binding")

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
INV, UNS, OK = B.OMNI_ERR_INVALID_ARG, B.OMNI_ERR_UNSUPPORTED, B.OMNI_OK


def weight_grad(dt=1, M=4, E=2, n=8, k=16, ws=None, nws=0, dw=FAKE):
    return B.lib().omni_expert_weight_grad(dt, M, E, n, k, M, M, FAKE, None, FAKE, None, FAKE, dw,
                                           ws, nws, None)


def test_tasks_of_a_weight_gradient():
    # a task's number rounded up to a stage or a part fits 31 bits
    for dt in (0, 1):
        assert weight_grad(dt, M=1 << 30) == B.OMNI_ERR_WORKSPACE
        assert weight_grad(dt, M=(1 << 30) + 1) == UNS
        assert weight_grad(dt, M=(1 << 31) - 1) == UNS


def test_experts_of_a_product():
    f = B.lib().omni_expert_matmul
    call = lambda E: f(1, 0, E, 8, 16, 0, 0, FAKE, None, FAKE, FAKE, 0, 0, FAKE, None, None)
    assert call(1 << 30) == OK
    assert call((1 << 30) + 1) == UNS
    assert call((1 << 31) - 1) == UNS
    g = B.lib().omni_quantized_expert_matmul
    call = lambda E: g(1, 0, E, 8, 16, 0, 0, FAKE, FAKE, None, FAKE, FAKE, FAKE, 0, FAKE, None,
                       None)
    assert call(1 << 30) == OK
    assert call((1 << 30) + 1) == UNS


def test_rows_of_a_combination():
    f = B.lib().omni_expert_combine
    # o missing ends a call whose size is taken
    call = lambda dt, L, K, n: f(dt, L, K, n, None, None, FAKE, 0, None)
    assert call(1, 1 << 23, 8, 8) == INV                  # 2^26 tasks
    assert call(1, (1 << 31) - 1, 1, 8) == UNS            # y of nearly 2^34 elements
    assert call(1, (1 << 31) - 128, 1, 8) == INV
    assert call(1, (1 << 31) - 127, 1, 8) == UNS
    assert call(0, 1, (1 << 31) - 1, 4) == INV
    assert call(0, (1 << 24) - 1, 127, 1 << 10) == INV    # y of 2^34 - 1024
    assert call(0, 1 << 24, 127, 1 << 10) == UNS


def test_tasks_of_the_backward_combination():
    f = B.lib().omni_expert_combine_backward
    call = lambda L, K, n: f(1, L, K, n, FAKE, FAKE, None, FAKE, FAKE, None)
    assert call((1 << 26) - 4, 1, 8) == INV               # dy missing
    assert call((1 << 26) - 3, 1, 8) == UNS
    assert call(1, (1 << 26) - 4, 8) == INV
    assert call(1 << 23, 8, 8) == UNS
    assert call(1 << 20, 8, 1 << 20) == INV               # the rows' length does not count


def test_rows_to_quantise():
    f = B.lib().omni_quantize_rows
    call = lambda R, k: f(1, R, k, None, FAKE, FAKE, None)
    assert call((1 << 26) - 4, 2048) == INV               # x missing
    assert call((1 << 26) - 3, 16) == UNS
    assert call((1 << 24) - 1, 2064) == INV
    assert call(1 << 24, 2064) == UNS


def test_tiles_of_a_weight_gradient():
    # launches of 2^32 work-items: tiles of up to 128 have 256, tiles of 256 have 512
    assert weight_grad(M=4, E=1 << 24, n=8, k=8) == UNS
    assert weight_grad(M=64 << 20, E=1 << 20, n=256, k=256 * 8) == UNS
