"""Failure detection of the 8-bit matrix product without a GPU fault.

Every wait inside its kernels is bounded.  A test-only copy of the library
(build.build_wait_test) makes the MMA warps wait, at their second group of 128
channels, for a barrier that nothing arrives on, with a limit of about 2 ms: each
role then gives up, copies and MMAs in flight are waited for, tensor memory is
released and the kernel returns.  gdr_linear_fp8_status reports it once, and the
regular library's next call on the same device is correct."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
TIMEOUT, OK, ERR_CUDA = 5, 0, 4


def _operands(rows, n, k):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randint(-4, 5, (rows, k), generator=g, device="cuda").float().to(torch.float8_e4m3fn)
    w = torch.randint(-4, 5, (n, k), generator=g, device="cuda").float().to(torch.float8_e4m3fn)
    return x, torch.ones(rows, -(-k // 128), device="cuda"), w, torch.ones(-(-n // 128), -(-k // 128), device="cuda")


# one kernel each: few tokens (K whole, K in parts), CTA pairs on 256 x 128 and on
# 256 x 256 tiles
@pytest.mark.parametrize("rows,n,k", [(3, 20000, 1024), (3, 256, 2048), (300, 4096, 2048), (1024, 8192, 1024)])
def test_a_wait_that_runs_out_is_reported_and_harmless(rows, n, k):
    import gated_delta_rule_150_b200 as gdr
    from gated_delta_rule_150_b200 import build as gdr_build
    gdr.lib()
    T = ctypes.CDLL(gdr_build.build_wait_test())
    for f in (T.gdr_linear_fp8, T.gdr_linear_fp8_status):
        f.restype = ctypes.c_int
    T.gdr_linear_fp8.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    T.gdr_linear_fp8_status.argtypes = [ctypes.c_void_p]
    ops = _operands(rows, n, k)
    plan = gdr.PreparedLinearFp8(*ops, out_dtype=torch.float32)
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert T.gdr_linear_fp8_status(st) == OK
    assert T.gdr_linear_fp8(ctypes.byref(plan.args), st) == OK
    torch.cuda.synchronize()
    assert T.gdr_linear_fp8_status(st) == TIMEOUT
    assert T.gdr_linear_fp8_status(st) == OK              # reported once
    y = plan.run()
    gdr.linear_fp8_status()
    assert torch.equal(y.double(), ops[0].double() @ ops[2].double().T)


def test_status_is_refused_while_capturing():
    import gated_delta_rule_150_b200 as gdr
    L = gdr.lib()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    keep = torch.zeros(4, device="cuda")
    with torch.cuda.graph(graph, stream=side):
        keep.add_(1)
        status = L.gdr_linear_fp8_status(ctypes.c_void_p(side.cuda_stream))
    assert status == ERR_CUDA
    graph.replay()
    torch.cuda.synchronize()
    gdr.linear_fp8_status()
