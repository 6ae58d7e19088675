"""The chunk kernels' wait of a whole warp: true for all lanes once every lane's barrier has
completed, false for all of them after its limit, with an error status. No fault, trap or hang."""
import ctypes
import os
import subprocess

import pytest
import torch

from paged_decode_attention_02_gb300 import binding, build_lib

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_warp_wait_runs_out_for_all_lanes(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = str(tmp_path / "libwarp_wait.so")
    subprocess.run([build_lib._nvcc(), *build_lib.ARCH, *build_lib.NVCC_FLAGS,
                    "-I" + os.path.join(build_lib.PKG, "csrc"), "-shared", "-o", path,
                    os.path.join(HERE, "cuda", "warp_wait_timeout.cu")], check=True)
    lib = ctypes.CDLL(path)
    for odd in (0, 1, 0):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        done = torch.full((32,), -1, dtype=torch.int32, device="cuda")
        elapsed = torch.zeros(1, dtype=torch.int64, device="cuda")
        rc = lib.pda_test_warp_wait(odd, *(ctypes.c_void_p(t.data_ptr())
                                           for t in (status, done, elapsed)),
                                    ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert rc == 0
        torch.cuda.synchronize()
        secs = int(elapsed.item()) / 1e9
        if odd:
            assert done.tolist() == [0] * 32
            assert int(status.item()) == binding.PDA_DEVERR_TIMEOUT
            assert 0.9 <= secs <= 5.0, secs
        else:
            assert done.tolist() == [1] * 32 and int(status.item()) == 0 and secs < 0.9
