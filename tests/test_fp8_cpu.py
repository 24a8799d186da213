"""The 8-bit projections without a GPU: pins of the oracle's format and formulas,
and the refusals of the C ABI and of the Python binding (which come before any
launch, so they need no device)."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_150_b200 as gdr
import oracle
from gated_delta_rule_150_b200 import build as gdr_build

bf16, f32, e4m3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# --- pins of the oracle ----------------------------------------------------------------------

def all_codes():
    t = torch.arange(256, dtype=torch.uint8).view(e4m3).double().numpy()
    return t[np.isfinite(t)]


def test_e4m3_keeps_every_code_and_rounds_ties_to_even():
    c = np.unique(np.abs(all_codes()))
    assert c.size == 127 and c[-1] == 448.0 and c[1] == 2.0 ** -9
    assert np.array_equal(oracle.e4m3(c), c) and np.array_equal(oracle.e4m3(-c), -c)
    mid = (c[:-1] + c[1:]) / 2
    got = oracle.e4m3(mid)
    even = np.where(np.arange(mid.size) % 2 == 0, c[:-1], c[1:])    # even code of each pair
    assert np.array_equal(got, even)
    assert np.array_equal(oracle.e4m3(mid * (1 + 1e-12)), c[1:])
    assert np.array_equal(oracle.e4m3(mid * (1 - 1e-12)), c[:-1])
    assert oracle.e4m3(np.array([1e9]))[0] == 448.0
    # torch's own conversion agrees on fp32 values inside the range
    x = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * 100
    x = x.clamp(-448, 448)
    assert np.array_equal(oracle.e4m3(x), x.to(e4m3).double().numpy())


def test_norm_pins():
    r = np.random.default_rng(2)
    x = r.standard_normal((5, 272))
    one = np.ones(272)
    codes, scale, h = oracle.norm_fp8(x, one, eps=0.0)
    assert codes.shape == (5, 272) and scale.shape == (5, 3) and np.array_equal(h, x)
    y = codes * np.repeat(scale, 128, axis=1)[:, :272]
    assert np.allclose(np.mean(y * y, axis=1), 1.0, rtol=1e-12)          # unit RMS
    assert np.allclose(np.abs(codes).reshape(5, -1).max(), 448.0)       # the largest is 448
    # the norm is of the sum, and a residual of zeros changes nothing
    a = oracle.norm_fp8(x, one, residual=np.zeros_like(x))
    assert all(np.array_equal(p, q) for p, q in zip(a, oracle.norm_fp8(x, one)))
    b = oracle.norm_fp8(x - 1.5, one, residual=np.full_like(x, 1.5))
    assert np.allclose(b[2], x, atol=1e-15)
    ref = torch.nn.functional.rms_norm(torch.from_numpy(x), (272,), torch.from_numpy(one), 1e-6).numpy()
    c, s, _ = oracle.norm_fp8(x, one)
    assert np.allclose(c * np.repeat(s, 128, axis=1)[:, :272], ref, rtol=1e-12)
    # zeros: the floor of the scale, codes 0
    c, s, _ = oracle.norm_fp8(np.zeros((1, 128)), np.ones(128))
    assert s[0, 0] == 1e-12 / 448 and not c.any()


def test_gated_norm_groups_run_over_the_heads():
    r = np.random.default_rng(3)
    o, g, w = r.standard_normal((4, 3, 64)), r.standard_normal((4, 3, 64)), r.standard_normal(64)
    codes, scale = oracle.gated_norm_fp8(o, g, w)
    y = oracle.output_epilogue(o, g, w).reshape(4, 192)
    assert scale.shape == (4, 2)
    assert np.allclose(scale[:, 0] * 448, np.abs(y[:, :128]).max(axis=1), rtol=1e-14)   # heads 0 and 1
    assert np.allclose(scale[:, 1] * 448, np.abs(y[:, 128:]).max(axis=1), rtol=1e-14)   # head 2
    assert np.allclose(codes * np.repeat(scale, 128, axis=1)[:, :192], y, rtol=1e-13)


def test_linear_is_the_product_of_what_the_codes_stand_for():
    r = np.random.default_rng(4)
    x, w = r.standard_normal((3, 160)), r.standard_normal((130, 160))
    xc, xs = oracle._scaled_rows(x)
    wc, ws = oracle.quantize_weight_fp8(w)
    assert ws.shape == (2, 2)
    y, size = oracle.linear_fp8(xc, xs, wc, ws)
    assert np.allclose(y, x @ w.T, rtol=1e-12, atol=1e-12)
    assert np.allclose(size, np.abs(x) @ np.abs(w).T, rtol=1e-12)


# --- refusals: C ABI -------------------------------------------------------------------------

@pytest.fixture(scope="module")
def L():
    gdr_build.build()
    return gdr.lib()


def _norm(**kw):
    a = gdr.NormFp8Args()
    a.rows, a.width, a.io_dtype, a.norm_eps = 4, 256, 0, 1e-6
    a.x, a.residual, a.norm_weight, a.residual_out, a.y, a.y_scale = (0x10000 * i for i in range(1, 7))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_norm_rejects_bad_arguments(L):
    call = lambda **kw: L.gdr_norm_fp8(ctypes.byref(_norm(**kw)), None)
    assert L.gdr_norm_fp8(None, None) == 1
    assert call(rows=-1) == 1 and call(rows=1 << 31) == 1
    assert call(width=0) == 1 and call(width=-16) == 1
    assert call(width=24) == 2 and call(width=32784) == 2
    assert call(io_dtype=2) == 1
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(norm_eps=eps) == 1
    assert call(residual=None) == 1                       # residual_out without residual
    for name in ("x", "norm_weight", "y", "y_scale"):
        assert call(**{name: None}) == 1, name
    for name in ("x", "residual", "norm_weight", "residual_out", "y"):
        assert call(**{name: 0x90008}) == 1, name
    assert call(y_scale=0x90002) == 1
    assert call(rows=0, x=None) == 0


def _gated(**kw):
    a = gdr.GatedNormFp8Args()
    a.rows, a.n_heads, a.d_v, a.o_dtype, a.gate_dtype, a.norm_eps = 4, 3, 64, 1, 0, 1e-6
    a.o, a.gate_raw, a.norm_weight, a.y, a.y_scale = (0x10000 * i for i in range(1, 6))
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_gated_norm_rejects_bad_arguments(L):
    call = lambda **kw: L.gdr_gated_norm_fp8(ctypes.byref(_gated(**kw)), None)
    assert L.gdr_gated_norm_fp8(None, None) == 1
    assert call(rows=-1) == 1 and call(rows=1 << 31) == 1 and call(n_heads=0) == 1
    assert call(d_v=32) == 2 and call(d_v=0) == 1
    assert call(n_heads=1 << 25, d_v=64) == 1             # H d_v past 32 bits
    assert call(o_dtype=5) == 1 and call(gate_dtype=-1) == 1 and call(norm_eps=-1.0) == 1
    for name in ("o", "gate_raw", "norm_weight", "y", "y_scale"):
        assert call(**{name: None}) == 1, name
    for name in ("o", "gate_raw", "norm_weight", "y"):
        assert call(**{name: 0x90004}) == 1, name
    assert call(rows=0, o=None) == 0


def test_quantize_rejects_bad_arguments(L):
    p = [ctypes.c_void_p(0x10000 * i) for i in range(1, 4)]
    call = lambda n=4, k=64, dt=0, w=p[0], c=p[1], s=p[2]: L.gdr_quantize_weight_fp8(n, k, dt, w, c, s, None)
    assert call(n=-1) == 1 and call(k=0) == 1 and call(k=40) == 2 and call(dt=3) == 1
    assert call(w=None) == 1 and call(c=None) == 1 and call(s=None) == 1
    assert call(w=ctypes.c_void_p(0x10008)) == 1 and call(c=ctypes.c_void_p(0x10001)) == 1
    assert call(n=0, w=None) == 0


def _linear(**kw):
    a = gdr.LinearFp8Args()
    a.rows, a.n, a.k, a.n_outs = 4, 200, 64, 2
    a.x, a.x_scale, a.w, a.w_scale = (0x10000 * i for i in range(1, 5))
    a.out_cols[0], a.out_cols[1] = 150, 50
    a.out_dtype[0], a.out_dtype[1] = 0, 1
    a.out[0], a.out[1] = 0x50000, 0x60000
    for k, v in kw.items():
        if isinstance(v, tuple):
            getattr(a, k)[v[0]] = v[1]
        else:
            setattr(a, k, v)
    return a


def test_linear_rejects_bad_arguments(L):
    call = lambda **kw: L.gdr_linear_fp8(ctypes.byref(_linear(**kw)), None)
    assert L.gdr_linear_fp8(None, None) == 1
    assert call(rows=-1) == 1 and call(rows=1 << 31) == 1
    assert call(n=0) == 1 and call(k=0) == 1 and call(k=72) == 2
    assert call(n_outs=0) == 1 and call(n_outs=9) == 1
    assert call(out_cols=(1, 51)) == 1 and call(out_cols=(1, 0)) == 1 and call(out_cols=(0, -150)) == 1
    assert call(out_dtype=(1, 2)) == 1
    for name in ("x", "x_scale", "w", "w_scale"):
        assert call(**{name: None}) == 1, name
    assert call(x=0x10008) == 1 and call(w=0x30008) == 1 and call(x_scale=0x20002) == 1
    assert call(out=(0, None)) == 1 and call(out=(0, 0x50001)) == 1 and call(out=(1, 0x60002)) == 1
    assert call(rows=0, x=None) == 0


# --- refusals: binding -----------------------------------------------------------------------

def _reaches_device_check(fn, *a, **kw):
    with pytest.raises(ValueError, match="CUDA tensors"):
        fn(*a, **kw)


def test_norm_binding():
    x, w = torch.zeros(3, 256, dtype=bf16), torch.ones(256)
    _reaches_device_check(gdr.norm_fp8, x, w)
    _reaches_device_check(gdr.norm_fp8, x, w, residual=x, residual_out=x)
    with pytest.raises(ValueError, match="2 dimensions"):
        gdr.norm_fp8(x[0], w)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        gdr.norm_fp8(x.half(), w)
    with pytest.raises(ValueError, match="multiple of 16"):
        gdr.norm_fp8(x[:, :24].contiguous(), w[:24])
    with pytest.raises(ValueError, match="multiple of 16"):
        gdr.norm_fp8(torch.zeros(1, 32784, dtype=bf16), torch.ones(32784))
    with pytest.raises(ValueError, match="norm_weight must have shape"):
        gdr.norm_fp8(x, w[:128])
    with pytest.raises(TypeError, match="norm_weight must be"):
        gdr.norm_fp8(x, w.bfloat16())
    with pytest.raises(TypeError, match="residual must be"):
        gdr.norm_fp8(x, w, residual=x.float())
    with pytest.raises(ValueError, match="needs a residual"):
        gdr.norm_fp8(x, w, residual_out=x)
    with pytest.raises(TypeError, match="out must be"):
        gdr.norm_fp8(x, w, out=torch.zeros(3, 256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="out_scale must have shape"):
        gdr.norm_fp8(x, w, out_scale=torch.zeros(3, 1))
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(ValueError, match="norm_eps"):
            gdr.norm_fp8(x, w, norm_eps=eps)


def test_gated_norm_binding():
    o, g, w = torch.zeros(3, 2, 64), torch.zeros(3, 2, 64, dtype=bf16), torch.ones(64)
    _reaches_device_check(gdr.gated_norm_fp8, o, g, w)
    with pytest.raises(ValueError, match="d_v must be"):
        gdr.gated_norm_fp8(o[..., :32].contiguous(), g, w)
    with pytest.raises(ValueError, match="one head"):
        gdr.gated_norm_fp8(o[:, :0], g[:, :0], w)
    with pytest.raises(ValueError, match="gate_raw must have shape"):
        gdr.gated_norm_fp8(o, g[:2], w)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        gdr.gated_norm_fp8(o, g.half(), w)
    with pytest.raises(ValueError, match="norm_weight must have shape"):
        gdr.gated_norm_fp8(o, g, torch.ones(128))


def test_quantize_binding():
    w = torch.zeros(5, 32)
    _reaches_device_check(gdr.quantize_weight_fp8, w)
    with pytest.raises(ValueError, match="multiple of 16"):
        gdr.quantize_weight_fp8(w[:, :24])
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        gdr.quantize_weight_fp8(w.double())
    with pytest.raises(ValueError, match="out_scale must have shape"):
        gdr.quantize_weight_fp8(w, out_scale=torch.zeros(1, 2))


def test_linear_binding():
    x, xs = torch.zeros(3, 144, dtype=e4m3), torch.zeros(3, 2)
    w, ws = torch.zeros(200, 144, dtype=e4m3), torch.zeros(2, 2)
    _reaches_device_check(gdr.linear_fp8, x, xs, w, ws)
    _reaches_device_check(gdr.linear_fp8, x, xs, w, ws, splits=(150, 50), out_dtype=(bf16, f32))
    with pytest.raises(TypeError, match="x must be"):
        gdr.linear_fp8(x.view(torch.uint8), xs, w, ws)
    with pytest.raises(ValueError, match="w must have shape"):
        gdr.linear_fp8(x, xs, w[:, :128].contiguous(), ws)
    with pytest.raises(ValueError, match="x_scale must have shape"):
        gdr.linear_fp8(x, xs.T.contiguous(), w, ws)
    with pytest.raises(ValueError, match="w_scale must have shape"):
        gdr.linear_fp8(x, xs, w, ws[:1])
    with pytest.raises(ValueError, match="K must be"):
        gdr.linear_fp8(x[:, :24].contiguous(), xs[:, :1], w[:, :24].contiguous(), ws[:, :1])
    with pytest.raises(ValueError, match="at least one row"):
        gdr.linear_fp8(x, xs, w[:0], ws[:0])
    for splits in ((), (150, 49), (0, 200), (25,) * 8 + (0,), (200, -1, 1)):
        with pytest.raises(ValueError, match="splits must be"):
            gdr.linear_fp8(x, xs, w, ws, splits=splits)
    with pytest.raises(TypeError, match="out_dtype"):
        gdr.linear_fp8(x, xs, w, ws, out_dtype=torch.float16)
    with pytest.raises(TypeError, match="out_dtype"):
        gdr.linear_fp8(x, xs, w, ws, splits=(100, 100), out_dtype=(bf16,))
    with pytest.raises(ValueError, match="one tensor for each"):
        gdr.linear_fp8(x, xs, w, ws, splits=(100, 100), out=torch.zeros(3, 200, dtype=bf16))
    with pytest.raises(ValueError, match=r"out\[0\] must have shape"):
        gdr.linear_fp8(x, xs, w, ws, out=torch.zeros(3, 100, dtype=bf16))


def test_outputs_must_lie_apart():
    buf = torch.zeros(64, dtype=f32)
    a, b = buf[:32], buf[16:48]
    with pytest.raises(ValueError, match="a must not overlap b"):
        gdr._need_apart([("a", a)], [("b", b)])
    with pytest.raises(ValueError, match="a must not overlap b"):
        gdr._need_apart([("a", a), ("b", b)], [])
    gdr._need_apart([("a", a)], [("b", buf[32:]), ("c", None), ("d", buf[:0])])
    gdr._need_apart([("a", a)], [("b", a)], same={("a", "b")})
    with pytest.raises(ValueError, match="overlap"):
        gdr._need_apart([("a", a)], [("b", b)], same={("a", "b")})
