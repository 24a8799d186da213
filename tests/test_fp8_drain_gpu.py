"""What a kernel of the 8-bit matrix product does after it gave up a bounded wait: it
waits, with a limit of its own, for everything it has in flight (tile loads, MMAs,
parts on their way to another CTA), releases its tensor memory and returns.

The test copy of the library lets one role stop at its second group of 128
channels.  Its error word then holds 1 (a wait was given up); 2 on top would say that
something in flight was not seen to end.  Nothing here hangs or faults the GPU."""
import ctypes
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
MMAS, LOADS, ODD_LOADS, SUMS, STORES, EVEN_LOADS = range(6)
TIMEOUT, OK = 5, 0


@pytest.fixture(scope="module")
def libs():
    import gated_delta_rule_150_b200 as gdr
    from gated_delta_rule_150_b200 import build as gdr_build
    gdr.lib()
    T = ctypes.CDLL(gdr_build.build_wait_test())
    for f in (T.gdr_linear_fp8, T.gdr_linear_fp8_status, T.gdr_linear_fp8_test_role, T.gdr_linear_fp8_test_word):
        f.restype = ctypes.c_int
    T.gdr_linear_fp8.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    T.gdr_linear_fp8_status.argtypes = [ctypes.c_void_p]
    yield gdr, T
    assert T.gdr_linear_fp8_test_role(MMAS) == 0          # as the other tests expect it


def _stop(libs, role, rows, n, k):
    gdr, T = libs
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randint(-4, 5, (rows, k), generator=g, device="cuda").float().to(torch.float8_e4m3fn)
    w = torch.randint(-4, 5, (n, k), generator=g, device="cuda").float().to(torch.float8_e4m3fn)
    plan = gdr.PreparedLinearFp8(x, torch.ones(rows, -(-k // 128), device="cuda"), w,
                                 torch.ones(-(-n // 128), -(-k // 128), device="cuda"), out_dtype=torch.float32)
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert T.gdr_linear_fp8_test_role(role) == 0
    torch.cuda.synchronize()
    assert T.gdr_linear_fp8_test_word() in (0, 1)
    took = []
    for _ in range(2):                                    # the first call also loads the kernel
        t0 = time.monotonic()
        assert T.gdr_linear_fp8(ctypes.byref(plan.args), st) == OK
        torch.cuda.synchronize()
        took.append(time.monotonic() - t0)
        assert T.gdr_linear_fp8_test_word() == 1          # given up, and all of it seen to end
    assert min(took) < 1.0                                # a wait for what never comes takes two seconds
    assert T.gdr_linear_fp8(ctypes.byref(plan.args), st) == OK
    torch.cuda.synchronize()
    assert T.gdr_linear_fp8_status(st) == TIMEOUT and T.gdr_linear_fp8_status(st) == OK
    y = plan.run()
    gdr.linear_fp8_status()
    assert torch.equal(y.double(), x.double() @ w.double().T)


# fewer groups than stages (all loads are issued before anything stops), more of them,
# K in parts, and each token tile
WHOLE = [(3, 20000, 256), (3, 20000, 1536), (64, 20000, 1024)]
PARTS = [(3, 256, 2048), (30, 512, 4096), (50, 512, 4096), (130, 1024, 4096)]


@pytest.mark.parametrize("rows,n,k,role", [(*c, r) for c in WHOLE for r in (MMAS, LOADS, SUMS)] +
                         [(*c, r) for c in PARTS for r in (MMAS, LOADS, ODD_LOADS, SUMS)])
def test_few_tokens(libs, rows, n, k, role):
    _stop(libs, role, rows, n, k)


# CTA pairs on 256 x 128 and on 256 x 256 tiles, one tile or several a pair.  Where one
# CTA of a pair stops loading, the other is up to all stages ahead of it.
@pytest.mark.parametrize("role", [MMAS, LOADS, ODD_LOADS, SUMS, STORES, EVEN_LOADS])
@pytest.mark.parametrize("rows,n,k", [(300, 4096, 256), (300, 4096, 2048), (1024, 8192, 256), (1024, 8192, 1024),
                                      (9000, 2048, 128), (2100, 1000, 4096)])
def test_cta_pairs(libs, rows, n, k, role):
    _stop(libs, role, rows, n, k)
