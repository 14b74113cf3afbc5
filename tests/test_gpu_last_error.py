"""A call that the runtime refuses returns its status once: the calls after it are as good as
without it."""
import ctypes

import pytest
import torch

from deepseek_sequential_mtp_gb300 import lib, synth

pytestmark = pytest.mark.gpu


def test_a_refused_call_does_not_fail_the_next_one():
    """Reading the error word of a stream that is being captured is refused (it would wait for
    the stream)."""
    cudart = ctypes.CDLL("libcudart.so.13")
    c = {k: v.cuda() for k, v in synth.make_verify_inputs(synth.VerifyConfig(name="v", R=4, gamma=2, V=500), 1).items()}
    call = lambda: lib.spec_verify(c["p"], c["q"], c["draft"], 7, 1)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    assert cudart.cudaStreamBeginCapture(handle, 2) == 0  # relaxed: other streams are not concerned
    with pytest.raises(lib.MtpError):
        lib.check_errors(side)
    cudart.cudaStreamEndCapture(handle, ctypes.byref(graph))
    cudart.cudaGetLastError()
    got = call()
    lib.check_errors()
    assert all(torch.equal(got[k], want[k]) for k in want)
