"""csrc/host_call.cpp: the check of tensors and the passing of arguments.  CPU only: no
tensor here is on a device, so that fits() never holds for one, and the entry points
are called with arguments that they refuse."""
import ctypes

import pytest
import torch

from cartesian_routed_atomic_amd import binding as B

H = B._load_host()
F32, BF = torch.float32, torch.bfloat16


def test_fits_wants_tensors_on_the_device():
    t = torch.zeros(2, 3)
    assert H.fits(0) and H.fits(0, None, F32, (2, 3)) and H.fits(0, None, None, None)
    for dev in (0, -1):
        assert not H.fits(dev, t, F32, (2, 3))
        assert not H.fits(dev, None, F32, (1,), t, F32, (2, 3))
    for bad in ((t, BF, (2, 3)), (t, F32, (2,)), (t, F32, [2, 3]), (t, "f32", (2, 3)),
                (7, F32, (2, 3)), (t, None, (2, 3))):
        assert not H.fits(0, *bad)
    with pytest.raises(TypeError):
        H.fits(0, t, F32)
    with pytest.raises(TypeError):
        H.fits("0", t, F32, (2, 3))


def test_entry_points_pass_what_they_are_given():
    rows = B._entries["omni_microscale_rows"]
    assert rows(1, 0, 64, None, None, None, None) == B.OMNI_OK
    assert rows(1, 4, 48, 64, 64, 64, None) == B.OMNI_ERR_UNSUPPORTED
    assert rows(1, 4, 64, None, 64, 64, 0) == B.OMNI_ERR_INVALID_ARG
    assert rows(1, 4, 64, torch.zeros(0), 64, 64, 0) == B.OMNI_ERR_INVALID_ARG
    route = B._entries["omni_expert_route"]
    ok = [1, 0, 8, 2, None, None, 0, 1, 1, 1, 1, 1.0, None, None, None, None]
    assert route(*ok) == B.OMNI_OK
    for at, value in ((11, float("inf")), (11, float("nan")), (3, 0), (1, -1)):
        assert route(*(ok[:at] + [value] + ok[at + 1:])) == B.OMNI_ERR_INVALID_ARG
    assert route(*(ok[:11] + [3] + ok[12:])) == B.OMNI_OK  # a whole number for a float


@pytest.mark.parametrize("args", [
    (1, 0, 64, None, None, None), (1, 0, 64, None, None, None, None, None),
    (1, 2 ** 31, 64, None, None, None, None), (1, -2 ** 31 - 1, 64, None, None, None, None),
    (1, 2 ** 70, 64, None, None, None, None), (1.5, 0, 64, None, None, None, None),
    (1, 0, "64", None, None, None, None), (1, 0, 64, "x", None, None, None),
    (1, 0, 64, 2 ** 70, None, None, None)])
def test_entry_points_refuse_what_they_cannot_pass(args):
    with pytest.raises((TypeError, OverflowError)):
        B._entries["omni_microscale_rows"](*args)


def test_entries_are_the_librarys():
    with pytest.raises(KeyError):
        H.entry("omni_abi_version", 1)
    address = ctypes.cast(B.lib().omni_expert_route, ctypes.c_void_p).value
    again = H.entry("omni_expert_route", address)
    assert again.__self__ == address == B._entries["omni_expert_route"].__self__


def test_tensors_without_memory_of_their_own():
    """Refused or told apart, without a C++ exception out of the module."""
    odd = [torch.eye(4).to_sparse(), torch.eye(4).to_sparse_csr(),
           torch.nested.nested_tensor([torch.zeros(2), torch.zeros(3)]),
           torch.zeros(4, 4, device="meta")]
    for t in odd:
        assert not H.fits(0, t, F32, (4, 4))
    for t in odd[:2]:
        with pytest.raises(TypeError):
            B._entries["omni_microscale_rows"](1, 0, 64, t, None, None, None)
    for t in odd[:2]:
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            B.microscale_rows(t)
