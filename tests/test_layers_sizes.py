"""Sizes of group norm far beyond any memory, asked for on the host: every size that the checks
accept has a plan, and a C entry point never ends the process."""
import os
import subprocess
import sys

import pytest

import transposed_convolution_amd as T

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = (0, 1, 4)  # float32, float16, bfloat16

SIZES = """
import ctypes, sys
import transposed_convolution_amd as T
shape, groups = tuple(int(s) for s in sys.argv[1].split(",")), int(sys.argv[2])
for dtype in (0, 1, 4):
    for backward in (0, 1):
        n = ctypes.c_size_t(0)
        st = T.load_library().group_norm_workspace_size(dtype, len(shape) - 2, T._i64(shape), groups, backward, ctypes.byref(n))
        print(st, n.value)
"""


@pytest.fixture(scope="module", autouse=True)
def library():
    if not os.path.exists(T.library_path()):
        from transposed_convolution_amd import build
        build.build()
    T.load_library()


@pytest.mark.parametrize("shape,groups", [
    ((1, 1, 1 << 50), 1), ((1, 1, 1 << 56), 1), ((1, 8, 1 << 53), 1), ((2, 8, 1 << 20, 1 << 16, 1 << 18), 4),
    ((3, 1 << 20, 1 << 36), 1 << 10), ((1, 257, 1 << 49), 257), ((1, 3, (1 << 56) + 1), 1), ((1, 1 << 26, 1 << 31), 2),
])
def test_workspace_of_sizes_beyond_any_memory(shape, groups):
    """The number of tiles of a chunk does not fit 32 bits here.  In a process of its own."""
    r = subprocess.run([sys.executable, "-c", SIZES, ",".join(map(str, shape)), str(groups)], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    elements = 1
    for s in shape:
        elements *= s
    lines = [tuple(map(int, line.split())) for line in r.stdout.splitlines()]
    assert len(lines) == 2 * len(TYPES)
    for status, size in lines:
        # a pair of float32 sums for each element at most, and room for the alignment
        assert status == 0 and 0 < size <= 8 * elements + (1 << 16), (status, size)


def _workspace(shape, groups, backward, dtype=1):
    import ctypes
    n = ctypes.c_size_t(0)
    return T.load_library().group_norm_workspace_size(dtype, len(shape) - 2, T._i64(shape), groups, backward, ctypes.byref(n))


@pytest.mark.parametrize("shape,groups", [
    (((1 << 21) + 5, 2, 2), 1), ((700000, 128, 1), 32), (((1 << 20) + 1, 64, 4), 16), ((1 << 22, 8, 1), 8), ((40000, 4096, 1), 64),
])
def test_many_images_are_served(shape, groups):
    assert _workspace(shape, groups, 0) == 0 and _workspace(shape, groups, 1) == 0


def test_launches_too_large_are_refused():
    """Forward 2^31 threads are 2^22 blocks of 512; the gradient's blocks have 256, and one for each
    16 channels makes the parameters' gradients, those of an empty x too."""
    for shape, groups, backward in ((((1 << 22) + 1, 8, 1), 8, 0), (((1 << 23) + 1, 8, 1), 8, 1), ((1, (1 << 27) + 16, 1), 1, 1),
                                    ((0, 1 << 30, 4), 1, 1), ((1, (1 << 30) + 1, 1), 1, 0)):
        assert _workspace(shape, groups, backward) == 3, shape
        assert T.convtranspose_last_error()
    lib, shape = T.load_library(), T._i64((0, 1 << 30, 4))
    assert lib.group_norm_backward_nd(1, 1, None, None, shape, 1, None, None, 0, None, None, 0, 0.0, 0.0, 0.0, 0, 0, None, None,
                                      256, 256, None, 0, None) == 3
