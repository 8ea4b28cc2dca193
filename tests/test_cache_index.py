"""The cache's index arithmetic against whole numbers of any size, on the host."""
import ctypes
import os
import shutil
import subprocess

import pytest

from diffusion_long_context_b200.build import CSRC


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = tmp_path_factory.mktemp("index")
    src = out / "index.cpp"
    src.write_text('#include "cache_index.cuh"\n'
                   'extern "C" int stored(int len, int j, int ps, int vs) { return focus::stored_vectors(len, j, ps, vs); }\n')
    so = out / "index.so"
    subprocess.run([shutil.which("g++"), "-O2", "-fwrapv", "-shared", "-fPIC", "-std=c++17", "-I" + CSRC, "-o", os.fspath(so),
                    os.fspath(src)], check=True)
    return ctypes.CDLL(os.fspath(so))


@pytest.mark.parametrize("page_shift", [4, 5, 6, 7])
@pytest.mark.parametrize("vec_shift", [3, 4])
def test_a_store_reads_no_row_behind_the_sequence(lib, page_shift, vec_shift):
    page = 1 << page_shift
    top = 2 ** 31 - page                                        # positions of the longest input
    for L in (1, 17, 300, 2 ** 27 - 1, 2 ** 27 + 69, 2 ** 28 + 5, 2 ** 30 + 77, top):
        cols = -(-L // page)
        pages = {0, 1, cols // 3, cols // 2, cols - 2, cols - 1}
        pages |= {cols - 1 - (2 ** s >> page_shift) for s in range(20, 31)}
        for j in (j for j in pages if 0 <= j < cols):
            for n in {0, 1, 5, L // 2, L - 1, L}:
                want = max(0, min(page, n - j * page)) << vec_shift
                assert lib.stored(n, j, page_shift, vec_shift) == want, (L, j, n)
