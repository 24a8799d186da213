"""Which code a value gets, bit by bit: the scale is the fp32 quotient max |y| / 448, a
weight's code is that of the fp32 quotient y / scale, and an activation's is that of
y / scale to 2^-21 of its size (1 / scale to 2 ulp and one product), so either
neighbour where y / scale is that close to the border between two codes.

The norms get rows whose y are known exactly: h = +-1 with eps 0 has the mean square 1,
and a gate of 200 the sigmoid 1, so y is the norm weight with a sign."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
bf16, f32, e4m3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gdr():
    import gated_delta_rule_150_b200 as m
    m.lib()
    return m


def _near_borders(rng, count, top):
    """fp32 values under the largest value `top` whose quotient by top / 448 lies on a
    border between two codes or a few fp32 steps beside it."""
    codes = np.unique(np.abs(torch.arange(256, dtype=torch.uint8).view(e4m3).double().numpy()[:127]))
    border = ((codes[:-1] + codes[1:]) / 2)[rng.integers(0, codes.size - 1, count)]
    scale = np.float32(top) / np.float32(448)
    y = (border * np.float64(scale)).astype(np.float32)
    for _ in range(3):
        y = np.where(rng.random(count) < 0.5, y, np.nextafter(y, np.float32(rng.choice([0, 3e38]))))
    y[0] = top
    return y.astype(np.float32), scale


def _assert_activation_codes(codes, scale, y, want_scale):
    """`y` [rows, width] exact, `want_scale` [rows, groups] of one value."""
    s = scale.cpu().numpy()
    assert np.array_equal(s, np.full_like(s, want_scale))
    q = y.astype(np.float64) / np.float64(want_scale)
    c = codes.double().cpu().numpy()
    assert ((c == oracle.e4m3(q * (1 - 2.0 ** -21))) | (c == oracle.e4m3(q * (1 + 2.0 ** -21)))).all()
    far = oracle.e4m3(q * (1 - 2.0 ** -21)) == oracle.e4m3(q * (1 + 2.0 ** -21))
    assert np.array_equal(c[far], oracle.e4m3(q)[far]) and not far.all()


@pytest.mark.parametrize("top", [448.0, 1.1, 3.7e-3, 5e9])
@pytest.mark.parametrize("rows,width", [(3, 128), (400, 128), (400, 256), (5, 2048), (500, 2048), (2, 16384)])
def test_norm(gdr, rows, width, top):
    rng = np.random.default_rng(width)
    groups = [_near_borders(rng, 128, top) for _ in range(width // 128)]
    w, scale = np.concatenate([g[0] for g in groups]), groups[0][1]
    sign = rng.choice([-1.0, 1.0], (rows, width)).astype(np.float32)
    for dt in (bf16, f32):
        c, s = gdr.norm_fp8(torch.from_numpy(sign).to(dt).cuda(), torch.from_numpy(w).cuda(), norm_eps=0.0)
        _assert_activation_codes(c, s, sign * w, scale)


@pytest.mark.parametrize("top", [448.0, 1.1, 3.7e-3, 5e9])
@pytest.mark.parametrize("rows,heads,d", [(3, 2, 64), (3, 3, 64), (70, 14, 64), (3, 1, 128), (70, 5, 128)])
def test_gated_norm(gdr, rows, heads, d, top):
    rng = np.random.default_rng(heads + d)
    w, scale = _near_borders(rng, d, top)
    sign = rng.choice([-1.0, 1.0], (rows, heads, d)).astype(np.float32)
    for o_dt, g_dt in ((bf16, bf16), (f32, bf16), (f32, f32)):
        c, s = gdr.gated_norm_fp8(torch.from_numpy(sign).to(o_dt).cuda(),
                                  torch.full((rows, heads, d), 200.0, device="cuda", dtype=g_dt),
                                  torch.from_numpy(w).cuda(), norm_eps=0.0)
        _assert_activation_codes(c, s, (sign * w).reshape(rows, -1), scale)


@pytest.mark.parametrize("dt", [bf16, f32])
@pytest.mark.parametrize("n,k", [(1, 16), (127, 400), (300, 1040), (3598, 896)])
def test_weights_scale_is_the_fp32_quotient(gdr, n, k, dt):
    """And not the product with a rounded 1 / 448, which is one step off in two blocks of
    five."""
    w = (0.03 * torch.randn(n, k, generator=torch.Generator(device="cuda").manual_seed(n + k), device="cuda")).to(dt)
    c, s = gdr.quantize_weight_fp8(w)
    pad = torch.nn.functional.pad(w.float(), (0, -k % 128, 0, -n % 128))
    top = pad.view(-(-n // 128), 128, -(-k // 128), 128).abs().amax((1, 3)).cpu().numpy()
    assert np.array_equal(s.cpu().numpy(), top / np.float32(448))
    each = s.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k].cpu().numpy()
    q = w.float().cpu().numpy() / each                         # fp32 division
    assert np.array_equal(c.double().cpu().numpy(), oracle.e4m3(q))


def test_squares_past_fp32_give_zeros(gdr):
    x = torch.randn(4, 256, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    x[1] *= 1e20
    y, s = gdr.norm_fp8(x, torch.ones(256, device="cuda"))
    assert not y[1].float().any() and (s[1].cpu().numpy() == np.float32(1e-12) / np.float32(448)).all()
    assert y[0].float().any() and torch.isfinite(y.float()).all()
    o = x.view(4, 4, 64).clone()
    y, s = gdr.gated_norm_fp8(o, torch.zeros_like(o), torch.ones(64, device="cuda"))
    assert not y[1].float().any() and y[2].float().any() and torch.isfinite(y.float()).all()
