"""The native tensor descriptors (_pydesc) are those of the Python binding,
byte for byte (CPU only)."""
import ctypes
import threading

import pytest
import torch

from mamba_ssd_scan_05_amd import ssd

pydesc = pytest.importorskip("mamba_ssd_scan_05_amd._pydesc")

TENSORS = [torch.zeros(2, 3, 4)[:, 1:], None, torch.zeros(5, dtype=torch.bool), torch.zeros(0, 3, dtype=torch.float16),
           torch.zeros(2, dtype=torch.int64), torch.zeros(1, 2, 3, 4, dtype=torch.bfloat16).transpose(1, 3),
           torch.tensor(3.0), torch.zeros(4, 1).expand(4, 9), torch.zeros(7, dtype=torch.uint8)[3:],
           torch.zeros(3, dtype=torch.int32), torch.zeros(6, requires_grad=True), torch.nn.Parameter(torch.zeros(2, 2))]


def raw(addrs):
    return [None if a is None else ctypes.string_at(a, ctypes.sizeof(ssd.SsdTensor)) for a in addrs]


def test_same_descriptors():
    buf, want = ssd._descs_py(*TENSORS)
    _, got = ssd._descs_native(*TENSORS)
    assert raw(got) == raw(want)
    assert ssd._descs is ssd._descs_native


def test_refusals():
    with pytest.raises(ValueError):
        pydesc.pack(torch.zeros(1, 1, 1, 1, 1))
    with pytest.raises(TypeError):
        pydesc.pack(torch.zeros(1), 3.0)
    with pytest.raises(ValueError):
        pydesc.pack(*[None] * 33)
    assert pydesc.pack() == ()


def test_threads_have_their_own():
    ready, done = threading.Event(), threading.Event()
    got = {}

    def other():
        got["a"] = pydesc.pack(torch.zeros(9, 9))
        got["raw"] = raw(got["a"])
        ready.set()
        done.wait(10)
        got["later"] = raw(got["a"])

    th = threading.Thread(target=other)
    th.start()
    ready.wait(10)
    mine = pydesc.pack(torch.zeros(1))
    done.set()
    th.join()
    assert mine[0] != got["a"][0] and got["later"] == got["raw"]


@pytest.mark.parametrize("descs", [ssd._descs_native, ssd._descs_py], ids=["native", "python"])
def test_a_call_in_between_leaves_the_descriptors_alone(descs):
    # a signal handler or a finalizer may call the library between a call's
    # descriptors and its C call
    keep, d = descs(torch.zeros(2, 3), None, torch.zeros(4, dtype=torch.bfloat16))
    before = raw(d)
    keep2, d2 = descs(torch.zeros(7, 7, 7), torch.zeros(1), torch.zeros(5, 1))
    assert raw(d) == before and raw(d2) != before


def test_the_library_reads_the_descriptors():
    # shapes and strides as the C side sees them, by what it refuses
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    for descs in (ssd._descs_native, ssd._descs_py):
        keep, d = descs(f(3, 24), f(3, 24), f(3, 24), f(3, 23), f(24), None, None, None, f(3, 24), f(3, 24))
        assert ssd.lib().ssd_glr_step(*d, None) == 2
        assert "i: dim 1 is 23, expected 24" in ssd.ssd_last_error()
