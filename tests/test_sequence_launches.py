"""What the sequence operators' entry points hand to their kernels, looked at on the host with
the launches replaced (launch_recorder.cu); no GPU needed, the pointers are never
dereferenced."""
import ctypes
import os
import subprocess

import pytest

from segmented_associative_scan_gb300 import buildlib
from segmented_associative_scan_gb300 import sequence as seq
from test_sequence_refusals import OK, fake, scan

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("recorder") / "recorder.so")
    subprocess.run([buildlib.nvcc(), *buildlib.ARCH, *buildlib.FLAGS, "-shared", "-Xlinker",
                    "-Bsymbolic", os.path.join(HERE, "launch_recorder.cu"), "-o", so], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(so)
    for name, (args, res) in seq.SIGNATURES.items():
        getattr(lib, name).argtypes, getattr(lib, name).restype = args, res
    lib.recorded_steps.restype = seq.Steps
    return lib


@pytest.mark.parametrize("suffix,elem", [("", 4), ("_bf16", 2), ("_fp16", 2)])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("N,T,row,step", [
    (4, 1, 8 * 1027, 1027),    # the first step of every row of a wider buffer
    (1, 64, 3, 32),            # the first row of a buffer whose rows lie anywhere
    (1, 1, 5, 7),
    (4, 64, 64 * 32, 32),
])
def test_16_byte_copies_start_on_16_byte_boundaries(recorder, suffix, elem, backward, N, T, row,
                                                    step):
    """The scan kernels form the addresses of a whole tile of steps, those past the row too: a
    copy of 16 bytes needs each of them aligned, also where it reads nothing."""
    at = lambda i: seq.Steps(fake(i), row, step)
    p = scan(N=N, T=T, x=at(1), dt=at(2), z=at(3),
             rows=seq.Rows(None, None, 0, None))
    if backward:
        g = seq.ScanGrads(at(13), None, fake(20), at(21), at(22), at(23),
                          seq.Steps(fake(24), 64 * 16, 16), seq.Steps(fake(25), 64 * 16, 16),
                          fake(26), fake(27), fake(28), fake(29))
        used = (0, 1, 2, 4, 5, 6, 7)
        fn = getattr(recorder, "rlca_selective_scan_backward" + suffix)
        status = fn(ctypes.byref(p), ctypes.byref(g), fake(40), 1 << 22, None)
    else:
        used = (0, 1, 2, 3)
        fn = getattr(recorder, "rlca_selective_scan" + suffix)
        status = fn(ctypes.byref(p), at(13), None, None, fake(40), 1 << 22, None)
    assert status == OK
    assert recorder.recorded_vec()  # every element that is read allows them
    for which in used:
        a = recorder.recorded_steps(which)
        for n in range(N):
            for t in range(32):  # steps of a tile, at the most
                assert (a.ptr + (n * a.row + t * a.step) * elem) % 16 == 0, (which, n, t)
