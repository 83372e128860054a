"""The gated recurrence's wait for the tiles before: what a tile gets from a tile that has published its state, and that a wait
which runs out (about a second, for a tile that publishes nothing) is flagged and leaves NaN, not a state that could be
taken for one."""
import ctypes
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu
ERR_TIMEOUT = 2  # device error word
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def look_back(tmp_path_factory):
    assert torch.cuda.is_available(), "the gpu-marked tests need a CUDA device"
    from linearized_attention_rope_gb300 import build

    lib = str(tmp_path_factory.mktemp("look_back") / "look_back_check.so")
    subprocess.run([build.NVCC, *build.ARCH, *build.FLAGS, "-I", build.CSRC, "-shared", "-o", lib,
                    os.path.join(HERE, "look_back_check.cu"), "-lcudart_static", "-lrt", "-ldl", "-lpthread"], check=True)
    fn = ctypes.CDLL(lib).look_back_check
    fn.argtypes, fn.restype = [ctypes.c_int] + [ctypes.c_void_p] * 4, ctypes.c_int

    def run(pairs, words):
        c = torch.full((32, 2 * pairs), 7.0, device="cuda")
        err = torch.zeros(4, dtype=torch.int32, device="cuda")
        st = torch.cuda.current_stream().cuda_stream
        assert fn(pairs, words.data_ptr(), c.data_ptr(), err.data_ptr(), st) == 0
        torch.cuda.synchronize()
        return c.cpu(), int(err[0])

    return run


@pytest.mark.parametrize("pairs", [1, 2])
def test_a_published_state_is_taken(look_back, pairs):
    want = torch.randn(32, 2 * pairs, generator=torch.Generator().manual_seed(1))
    words = torch.zeros(192 * pairs, dtype=torch.int64)
    words[:64 * pairs] = (want.view(torch.int32).long() & 0xffffffff | 1 << 32).reshape(-1)
    c, err = look_back(pairs, words.cuda())
    assert err == 0 and torch.equal(c, want)


@pytest.mark.parametrize("pairs", [1, 2])
def test_a_wait_that_runs_out_leaves_nan(look_back, pairs):
    c, err = look_back(pairs, torch.zeros(192 * pairs, dtype=torch.int64, device="cuda"))
    assert err == ERR_TIMEOUT and c.isnan().all()
