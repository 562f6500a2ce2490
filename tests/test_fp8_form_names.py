"""The kernels of the 8-bit products that the library holds, and sizes that run on each of them
(tests/test_fp8_every_form_gpu.py calls them; here without a GPU)."""
import re
import shutil
import subprocess

import pytest

from invariant_bi_rmsnorm_gb300 import _lib

# form (include/bi.h, bi_gemm_fp8_form) -> rows of x, rows of W, K: three parts of K or five, rows and
# columns that end inside a tile
FORMS = {
    1128007: (65, 136, 2064), 1256005: (520, 3208, 2064),
    2016205: (7, 24840, 2064), 2032205: (27, 15368, 2064), 2064204: (37, 19464, 2064), 2128204: (100, 19464, 4112),
    3016103: (3, 12424, 2064), 3016104: (3, 5896, 2064), 3016108: (3, 136, 2064),
    3016202: (7, 18952, 2064), 3016203: (3, 18952, 2064),
    3032103: (19, 12424, 2064), 3032104: (19, 5896, 2064), 3032108: (19, 136, 2064),
    3064103: (37, 5896, 2064), 3064106: (37, 136, 2064), 3128103: (520, 648, 4112), 3128106: (65, 136, 4112),
}
SWIGLU_FORMS = {
    1256006: (65, 288, 2064),
    2016205: (7, 24864, 2064), 2032205: (19, 15392, 2064), 2064204: (37, 19488, 2064), 2128204: (100, 19488, 4112),
    3016202: (7, 11808, 2064), 3016203: (3, 11808, 2064), 3016205: (3, 288, 2064),
    3032202: (19, 11808, 2064), 3032204: (19, 288, 2064), 3064202: (37, 7200, 4112), 3064204: (37, 288, 2064),
    3128204: (65, 288, 4112),
}


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return _lib.load()


def form_of(kernel, args):
    """(form without the ring's depth where the name does not say it, SwiGLU)."""
    if kernel == "parts":
        rows, tiles, swiglu, stages = args
        return 3000000 + 1000 * int(rows) + 100 * int(tiles) + int(stages), swiglu == "true"
    if kernel == "whole":
        return 2000000 + 1000 * int(args[0]), args[1] == "true"
    return 1000000 + 128000 * int(args[1]), args[0] == "true"


def test_every_kernel_of_the_library_has_its_sizes(lib):
    """And no kernel is in the library that no size runs on."""
    if shutil.which("nm") is None:
        pytest.skip("no nm")
    names = subprocess.run(["nm", "-C", _lib.LIB_PATH], capture_output=True, text=True, check=True).stdout
    held = {form_of(k, a.split(", ")) for k, a in re.findall(r"::gemm_fp8_(parts|whole|pair)_kernel<([^>]*)>\(", names)}
    listed = {(f if f >= 3000000 else f // 1000 * 1000, sw) for forms, sw in ((FORMS, False), (SWIGLU_FORMS, True)) for f in forms}
    assert held == listed


@pytest.mark.parametrize("M,N,K", [(0, 64, 64), (-1, 64, 64), (4, 4, 64), (4, 12, 64), (4, 64, 8), (4, 64, 72), (2 ** 31 - 1, 64, 64)])
def test_sizes_that_are_refused_have_no_form(lib, M, N, K):
    assert lib.bi_gemm_fp8_form(M, N, K, 0) == 0


def test_swiglu_sizes_that_are_refused_have_no_form(lib):
    import invariant_bi_rmsnorm_gb300 as bi
    assert bi.gemm_fp8_form(4, 16, 64, True) == bi.gemm_fp8_form(4, 48, 64, True) == 0
    assert bi.gemm_fp8_form(2 ** 32 + 4, 64, 64) == 0
