"""The tcgen05 key-weights kernel's bounded waits, running out (needs a GB300).

As in the attention kernels' test: a test variant of the library
(PKV_TEST_HOLD_ARRIVAL, a 20 ms wait limit) in which one epilogue warp can
withhold its release of an accumulator. The issuing warp's wait runs out, every
role unwinds, tensor memory is freed, the status bit is set, and the next call
through the same library is right."""
import ctypes
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

from paged_kv_cache_varlen_gb300 import binding, build

from .test_gpu_budget import Batch, i32, status_word

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hold_lib(tmp_path_factory):
    out = tmp_path_factory.mktemp("hold_budget")
    defines = ["-DPKV_TEST_HOLD_ARRIVAL", "-DPKV_WAIT_TIMEOUT_NS=20000000ull"]

    def comp(src):
        obj = str(out / (os.path.splitext(src)[0] + ".o"))
        subprocess.run([build.nvcc(), *build.NVCC_FLAGS, *defines, "-c",
                        os.path.join(build.CSRC, src), "-o", obj], check=True, capture_output=True)
        return obj

    with ThreadPoolExecutor(len(build.SOURCES)) as ex:
        objs = list(ex.map(comp, build.SOURCES))
    path = str(out / "libpkv_hold.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-shared", "-o", path, *objs, "-cudart", "static"],
                   check=True, capture_output=True)
    lib = binding.load_library(path)
    lib.pkv_test_hold_key_weights.restype = ctypes.c_int
    lib.pkv_test_hold_key_weights.argtypes = [ctypes.c_int]
    return lib


@pytest.mark.parametrize("max_len", [900, 1 << 20])  # a CTA for each item; a list of items
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(hold_lib, max_len):
    b = Batch([900, 600, 257], [300, 1, 200], 8, 2, 128, seed=41, poison=False)
    want = b.call(torch.zeros((3, 2, max_len), device="cuda"))
    table, cu, lens = i32(b.table), i32(b.cu), i32(b.lens)
    lse = torch.from_numpy(b.lse).cuda()

    def call():
        out, st = torch.zeros((3, 2, max_len), device="cuda"), status_word()
        status = hold_lib.pkv_attention_key_weights(
            out.data_ptr(), out.data_ptr(), b.q.data_ptr(), b.pool.data_ptr(), lse.data_ptr(),
            table.data_ptr(), table.shape[1], cu.data_ptr(), lens.data_ptr(), None, None, 3,
            max_len, 3, b.q.shape[0], 300, max_len, 8, 2, 128, 16, b.nb,
            float(np.float32(b.scale)), 1.0, st.data_ptr(),
            torch.cuda.current_stream().cuda_stream)
        assert status == 0
        torch.cuda.synchronize()
        return out, st.item()

    assert hold_lib.pkv_test_hold_key_weights(1) == 0
    try:
        _, status = call()
    finally:
        assert hold_lib.pkv_test_hold_key_weights(0) == 0
    assert status == binding.DEV_TIMEOUT
    out, status = call()
    assert status == 0
    assert torch.equal(out, want)
