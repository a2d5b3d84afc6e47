"""Attention to the 8-bit cache at the edges of what its documentation allows."""
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import speculative_decoding_verification_36_gb300 as sv
from speculative_decoding_verification_36_gb300 import _lib
from test_gpu_kv8 import BF16, F32, attend, attend_case, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,dtype", [(4, BF16), (40, BF16), (200, BF16), (5, F32)])
def test_bad_parents_of_a_padded_sequence(T, dtype):
    """A parent outside [-1, i) makes all T rows of its sequence NaN, those of padding too, wherever it lies and
    however few tokens there are; padding of the other sequences stays."""
    rng = np.random.default_rng(T)
    for n_new in (0, 1, T - 1, T):
        for node, parent in ((T - 2, T - 2), (0, -2)):
            x = attend_case(rng, 4, T, 4, 2, 64, dtype, "int8", 16, 16, [64, 300, 5, 40], tree=True)
            x["n_new"] = np.array([n_new, 0, T, T // 2], np.int32)
            x["parents"][0, node] = parent
            out = torch.full(x["q"].shape, 5.0, dtype=dtype, device=x["q"].device)
            got = attend(x, out=out)
            assert sv.spec_get_status() == sv.SPEC_FLAG_BAD_DATA
            assert torch.isnan(got[0]).all()
            check(x, got, skip=[0])


@pytest.mark.parametrize("limit", [1, 31, 64, 2000])
def test_a_wait_that_ran_out_is_told_from_one_that_did_not(limit):
    """Also under limits that leave a wait one look: a complete phase is no timeout, one that stays open is, and
    later waits do not wait."""
    try:
        sv.spec_test_spin_limit(limit)
        assert sv.spec_test_attend_wait_probe() == (0, 1, 0)
    finally:
        sv.spec_test_spin_limit(0)
    assert sv.spec_get_status() == 0


def test_two_threads_whose_trees_differ(tmp_path):
    """Launches of one kernel with shared memory of different sizes, from two host threads."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    _lib.load()  # the library is built
    here = os.path.dirname(os.path.abspath(__file__))
    cuda, libdir = os.environ.get("CUDA_HOME", "/usr/local/cuda"), os.path.dirname(_lib.LIB_PATH)
    exe = str(tmp_path / "c_abi_threads")
    res = subprocess.run([cc, "-O2", "-std=c99", "-I", os.path.join(os.path.dirname(here), "include"), "-I", os.path.join(cuda, "include"),
                          os.path.join(here, "c_abi_threads.c"), "-o", exe, "-L", libdir, "-l:libspecverify.so", f"-Wl,-rpath,{libdir}",
                          "-L", os.path.join(cuda, "lib64"), "-lcudart", f"-Wl,-rpath,{os.path.join(cuda, 'lib64')}", "-lpthread"],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    res = subprocess.run([exe], capture_output=True, text=True, timeout=100)
    assert res.returncode == 0, (res.returncode, res.stderr)
