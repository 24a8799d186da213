"""A product beside a kernel that holds the tensor memory of every SM for longer than the
product's waits last: it waits for its columns, which is not a give-up, and is right.

The test copy of the library (waits of some 2 ms) launches the holder, which gives its
columns back after 20 ms."""
import ctypes
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
HOLD_NS = 20_000_000


@pytest.fixture(scope="module")
def libs():
    import gated_delta_rule_150_b200 as gdr
    from gated_delta_rule_150_b200 import build as gdr_build
    gdr.lib()
    T = ctypes.CDLL(gdr_build.build_wait_test())
    for f in (T.gdr_linear_fp8, T.gdr_linear_fp8_test_role, T.gdr_linear_fp8_test_word, T.gdr_test_hold_tmem):
        f.restype = ctypes.c_int
    T.gdr_linear_fp8.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    T.gdr_test_hold_tmem.argtypes = [ctypes.c_uint64, ctypes.c_void_p]
    assert T.gdr_linear_fp8_test_role(-1) == 0            # no role stops
    yield gdr, T
    assert T.gdr_linear_fp8_test_role(0) == 0


# token tiles of 16, 32 and 64; K whole with fewer groups than stages and with more, and in
# parts; CTA pairs, which do not fit beside the holder
@pytest.mark.parametrize("rows,n,k", [(3, 20000, 256), (3, 20000, 1536), (3, 256, 2048), (30, 512, 4096), (50, 512, 4096),
                                      (64, 20000, 1024), (300, 4096, 1024), (1024, 8192, 1024)])
def test_waiting_for_columns_is_no_give_up(libs, rows, n, k):
    gdr, T = libs
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randint(-4, 5, (rows, k), generator=g, device="cuda").float().to(torch.float8_e4m3fn)
    w = torch.randint(-4, 5, (n, k), generator=g, device="cuda").float().to(torch.float8_e4m3fn)
    plan = gdr.PreparedLinearFp8(x, torch.ones(rows, -(-k // 128), device="cuda"), w,
                                 torch.ones(-(-n // 128), -(-k // 128), device="cuda"), out_dtype=torch.float32)
    plan.outputs.fill_(float("nan"))
    holder, user = torch.cuda.Stream(), torch.cuda.Stream()
    assert T.gdr_linear_fp8(ctypes.byref(plan.args), ctypes.c_void_p(user.cuda_stream)) == 0     # loads the kernel
    torch.cuda.synchronize()
    plan.outputs.fill_(float("nan"))
    torch.cuda.synchronize()
    assert T.gdr_linear_fp8_test_word() in (0, 1)
    t0 = time.monotonic()
    assert T.gdr_test_hold_tmem(HOLD_NS, ctypes.c_void_p(holder.cuda_stream)) == 0
    time.sleep(0.002)
    assert T.gdr_linear_fp8(ctypes.byref(plan.args), ctypes.c_void_p(user.cuda_stream)) == 0
    user.synchronize()
    took = time.monotonic() - t0
    torch.cuda.synchronize()
    assert took > 0.9e-9 * HOLD_NS                        # it had to wait for the holder
    assert T.gdr_linear_fp8_test_word() == 0
    assert torch.equal(plan.outputs.double(), x.double() @ w.double().T)
