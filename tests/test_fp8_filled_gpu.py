"""The 8-bit projections into outputs that hold NaN before the call, over the shapes
where a remainder can go wrong, with comparisons that a NaN cannot pass: an element
that is not written, or written from a factor of NaN or 0 times infinity, fails.
The oracle and the bounds are those of test_fp8_gpu.py."""
import numpy as np
import pytest
import torch

import oracle
import test_fp8_gpu as base
from fp8_checks import U, assert_within, check_codes, check_linear, nan_filled

pytestmark = pytest.mark.gpu
bf16, f32, e4m3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
SCALE = 4e-6


@pytest.fixture(scope="module")
def gdr():
    import gated_delta_rule_150_b200 as m
    m.lib()
    return m


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _groups(n):
    return -(-n // 128)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dt", [bf16, f32])
@pytest.mark.parametrize("rows,width", [(5, w) for w in (16, 112, 128, 144, 896, 1024, 1040, 2048, 2064, 4096, 4112,
                                                         8192, 8208, 16384, 16400, 32768)] +
                         [(r, w) for r in (297, 303, 1001) for w in (16, 112, 128, 144, 272, 528, 1040, 2064)])
def test_norm(gdr, rows, width, dt, residual):
    g = _gen(rows + width)
    x = torch.randn(rows, width, generator=g, device="cuda").to(dt)
    r = (3 * torch.randn(rows, width, generator=g, device="cuda")).to(dt) if residual else None
    w = 1 + 0.1 * torch.randn(width, generator=g, device="cuda")
    out, s = nan_filled(rows, width, dtype=e4m3), nan_filled(rows, _groups(width), dtype=f32)
    h = nan_filled(rows, width, dtype=dt) if residual else None
    gdr.norm_fp8(x, w, residual=r, out=out, out_scale=s, residual_out=h)
    rc, rs, rh = oracle.norm_fp8(x, w, r)
    check_codes(out, s, rc, rs, SCALE, "norm")
    if residual:
        assert_within(h, rh, (2.0 ** -8 if dt == bf16 else U) * 1.01 * np.abs(rh), "sum")


@pytest.mark.parametrize("o_dt,g_dt", [(bf16, bf16), (f32, bf16), (f32, f32), (bf16, f32)])
@pytest.mark.parametrize("rows,heads,d", [(1, 1, 64), (1, 14, 64), (3, 3, 64), (257, 14, 64), (1, 1, 128), (5, 7, 128),
                                          (300, 32, 128), (2049, 1, 64), (77, 5, 64)])
def test_gated_norm(gdr, rows, heads, d, o_dt, g_dt):
    g = _gen(rows + heads + d)
    o = torch.randn(rows, heads, d, generator=g, device="cuda").to(o_dt)
    gate = (2 * torch.randn(rows, heads, d, generator=g, device="cuda")).to(g_dt)
    w = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    out, s = nan_filled(rows, heads * d, dtype=e4m3), nan_filled(rows, _groups(heads * d), dtype=f32)
    gdr.gated_norm_fp8(o, gate, w, out=out, out_scale=s)
    rc, rs = oracle.gated_norm_fp8(o, gate, w)
    check_codes(out, s, rc, rs, SCALE + (4 + 2.4 * float(gate.float().abs().max())) * U, "gated norm")


@pytest.mark.parametrize("dt", [bf16, f32])
@pytest.mark.parametrize("n,k", [(1, 16), (14, 896), (127, 128), (128, 144), (129, 16), (300, 1040), (3598, 896)])
def test_quantize_weight(gdr, n, k, dt):
    w = (0.05 * torch.randn(n, k, generator=_gen(n + k), device="cuda")).to(dt)
    out, s = nan_filled(n, k, dtype=e4m3), nan_filled(_groups(n), _groups(k), dtype=f32)
    gdr.quantize_weight_fp8(w, out=out, out_scale=s)
    check_codes(out, s, *oracle.quantize_weight_fp8(w), 3 * U, "weights")


def _codes(g, rows, width):
    return (60 * torch.randn(rows, width, generator=g, device="cuda")).clamp(-448, 448).to(e4m3)


def _operands(seed, rows, n, k):
    g = _gen(seed)
    scales = lambda r: (0.5 + torch.rand(r, _groups(k), generator=g, device="cuda")) / 64
    return _codes(g, rows, k), scales(rows), _codes(g, n, k), scales(_groups(n))


def _linear(gdr, rows, cols, kinds, k, lead=0):
    """A product into tensors of NaN that begin `lead` elements into their buffers,
    every element against the oracle (the first and last rows where there are many)."""
    n = sum(cols)
    ops = _operands(rows + 7 * n + k, rows, n, k)
    dts = [bf16 if c == "b" else f32 for c in kinds]
    outs = [nan_filled(rows * c + lead, dtype=t)[lead:].view(rows, c) for c, t in zip(cols, dts)]
    gdr.linear_fp8(*ops, splits=cols, out_dtype=dts, out=outs)
    gdr.linear_fp8_status()
    assert all(torch.isfinite(t).all() for t in outs)
    at = torch.arange(rows, device="cuda")
    if rows * n > 1 << 22:
        at = torch.cat([at[:70], at[-70:]])
    check_linear([t[at] for t in outs], oracle.linear_fp8(ops[0][at], ops[1][at], *ops[2:]), cols, k)


@pytest.mark.parametrize("dt", "bf")
@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 32, 33, 36, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 1000])
@pytest.mark.parametrize("n,k", [(896, 896), (3598, 896), (130, 144)])
def test_linear_rows(gdr, rows, n, k, dt):
    _linear(gdr, rows, (n,), dt, k)


@pytest.mark.parametrize("rows", [1, 40, 300, 2100])
@pytest.mark.parametrize("n", [1, 2, 14, 100, 127, 128, 129, 255, 256, 257, 640])
@pytest.mark.parametrize("k", [16, 128, 272, 1040])
def test_linear_columns_and_depths(gdr, rows, n, k):
    _linear(gdr, rows, (n,), "f", k)


@pytest.mark.parametrize("dt", "bf")
@pytest.mark.parametrize("rows", [700, 2100, 20000])
@pytest.mark.parametrize("n", [8, 132, 200, 264, 520, 776])
def test_linear_last_tile_partly_empty(gdr, rows, n, dt):
    _linear(gdr, rows, (n,), dt, 144)


@pytest.mark.parametrize("lead", [0, 3, 8])
@pytest.mark.parametrize("rows", [1, 20, 200, 1030, 4099])
@pytest.mark.parametrize("cols,kinds", [((896, 896, 896, 896, 14), "bbbff"), ((130, 3, 1), "bfb"), ((1, 255), "fb"),
                                        ((64,) * 8, "bfbfbfbf"), ((256, 257, 127), "fbf"), ((1001,), "b"), ((2050,), "f"),
                                        ((3, 14, 777, 5, 300, 1, 131, 260), "bfbbfbbf")])
def test_linear_splits(gdr, rows, cols, kinds, lead):
    _linear(gdr, rows, cols, kinds, 400, lead)


@pytest.mark.parametrize("name,args", [("test_mixer_layer_from_residual_stream_to_output", (3, 64, False)),
                                       ("test_mixer_layer_from_residual_stream_to_output", (2, 128, True)),
                                       ("test_decode_layer_on_fp32_outputs", ()),
                                       ("test_norm_zero_tiny_huge_and_non_finite_rows", ()),
                                       ("test_gated_norm_far_gates_and_zero_heads", ()),
                                       ("test_offsets_past_32_bits", ())])
def test_layers_special_rows_and_far_offsets(gdr, monkeypatch, name, args):
    """Whole runs of test_fp8_gpu.py with the comparisons of this file."""
    monkeypatch.setattr(base, "_check_codes", check_codes)
    monkeypatch.setattr(base, "_check_linear",
                        lambda outs, ops, cols, k: check_linear(outs, oracle.linear_fp8(*ops), cols, k))
    getattr(base, name)(gdr, *args)
