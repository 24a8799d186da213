"""The 8-bit projections on the GPU against the fp64 oracle.

Tolerances, derived from the arithmetic (u = 2^-24, half an fp32 step):

* scale of norm_fp8: the sum of squares is at most 64 fused multiply-adds in a
  thread, 5 warp shuffles and 16 warps' sums (85 u, halved by the square root),
  one rounding of h (u), rsqrtf (2 ulp = 4 u), the mean's division, two
  products and the division by 448 (4 u): under 54 u = 3.2e-6.  SCALE = 4e-6.
* gated_norm_fp8: the sums are shorter (16 products, 3 shuffles); the sigmoid adds
  the rounding of g log2 e (2 |g| u in the power, with the constant's), the 2-ulp
  power and reciprocal and three roundings, which the shorter sums make room for:
  SCALE + (4 + 2.4 |g|) u.
* a code: y / scale carries the error of y, of the scale's reciprocal (2 u) and
  one rounding more, together under twice the scale's tolerance, and is then
  rounded to e4m3: off by at most half a step of e4m3 at its size.
* residual_out: one rounding, 2^-8 of the value in bf16; in fp32 the sum itself,
  one u.
* quantize_weight_fp8: no arithmetic before the scale: two roundings.
* linear_fp8 in fp32: K products and the groups' sums in some order, each
  addition off by at most 2 u (the tensor core may truncate) of the sum of the
  terms' sizes: (K + groups + 8) 2 u sum |terms|; in bf16 2^-8 of the value
  on top.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
bf16, f32, e4m3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
SCALE = 4e-6


@pytest.fixture(scope="module")
def gdr():
    import gated_delta_rule_150_b200 as m
    m.lib()
    return m


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _np(t):
    return t.double().cpu().numpy()


def _check_codes(codes, scale, ref_codes, ref_scale, tol, what=""):
    s = _np(scale)
    assert s.shape == ref_scale.shape
    assert (np.abs(s - ref_scale) <= tol * ref_scale).all(), \
        f"{what} scale off by {np.max(np.abs(s / ref_scale - 1)):.2e}"
    t = np.abs(ref_codes) * (1 + 2 * np.max(tol))
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(t, 1e-30))), -6.0) - 3)
    off = np.abs(_np(codes) - ref_codes)
    bad = off > step / 2 + 2 * np.max(tol) * np.abs(ref_codes)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} codes out of bound"


def _check_norm(gdr, rows, width, dt, residual, seed=0):
    g = _gen(seed + 31 * rows + width)
    x = torch.randn(rows, width, generator=g, device="cuda").to(dt)
    r = (3 * torch.randn(rows, width, generator=g, device="cuda")).to(dt) if residual else None
    w = 1 + 0.1 * torch.randn(width, generator=g, device="cuda")
    got = gdr.norm_fp8(x, w, residual=r)
    torch.cuda.synchronize()
    rc, rs, h = oracle.norm_fp8(x, w, r)
    _check_codes(got[0], got[1], rc, rs, SCALE, "norm")
    assert len(got) == (3 if residual else 2)
    if residual:
        assert got[2].dtype == dt
        rel = 2.0 ** -8 if dt == bf16 else U
        assert (np.abs(_np(got[2]) - h) <= rel * 1.01 * np.abs(h)).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dt", [bf16, f32])
@pytest.mark.parametrize("width", [16, 112, 128, 144, 896, 1024, 1040, 2048, 2064, 4096, 4112, 8192, 8208, 16384, 32768])
def test_norm_widths(gdr, width, dt, residual):
    _check_norm(gdr, 5, width, dt, residual)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 127, 1000, 4099])
@pytest.mark.parametrize("width", [896, 2048, 4112])
def test_norm_rows(gdr, rows, width):
    _check_norm(gdr, rows, width, bf16, True, seed=1)


def test_norm_in_place_and_guards(gdr):
    """residual_out may be the residual or x itself; nothing past the outputs is written."""
    g = _gen(5)
    rows, width = 37, 912
    x = torch.randn(rows, width, generator=g, device="cuda").to(bf16)
    r = torch.randn(rows, width, generator=g, device="cuda").to(bf16)
    w = torch.ones(width, device="cuda")
    ref = gdr.norm_fp8(x, w, residual=r)
    for target in ("x", "residual"):
        a, b = x.clone(), r.clone()
        ybuf = torch.full(((rows + 2) * width,), 0x55, dtype=torch.uint8, device="cuda")
        sbuf = torch.full(((rows + 2) * 8,), -7.0, device="cuda")
        y = ybuf[width:width * (rows + 1)].view(rows, width).view(e4m3)
        s = sbuf[8:8 * (rows + 1)].view(rows, 8)
        got = gdr.norm_fp8(a, w, residual=b, residual_out=a if target == "x" else b, out=y, out_scale=s)
        assert got[2] is (a if target == "x" else b)
        assert torch.equal(got[2], ref[2]) and torch.equal(s, ref[1])
        assert torch.equal(y.view(torch.uint8), ref[0].view(torch.uint8))
        assert (ybuf[:width] == 0x55).all() and (ybuf[width * (rows + 1):] == 0x55).all()
        assert (sbuf[:8] == -7).all() and (sbuf[8 * (rows + 1):] == -7).all()


def test_norm_zero_tiny_huge_and_non_finite_rows(gdr):
    rows, width = 6, 400
    x = torch.randn(rows, width, generator=_gen(6), device="cuda")
    x[0] = 0
    x[1] *= 1e-18                 # squares vanish beside eps
    x[2] *= 1e15
    x[3, 5] = float("nan")
    x[4, 390] = float("inf")      # last, shorter group
    w = torch.ones(width, device="cuda")
    y, s = gdr.norm_fp8(x, w)
    y, s = _np(y), _np(s)
    assert not y[0].any() and (np.abs(s[0] - 1e-12 / 448) <= 1e-7 * s[0]).all()
    rc, rs, _ = oracle.norm_fp8(x[1:3], w)
    assert np.allclose(s[1:3], rs, rtol=SCALE)
    assert np.isnan(s[3]).all() and np.isnan(y[3]).all()          # the mean is NaN
    # an infinite mean: 0 for finite values, NaN for the infinite one, whose group it takes along
    assert np.isnan(s[4, 3]) and np.isnan(y[4, 384:]).all()
    assert not y[4, :384].any() and np.allclose(s[4, :3], 1e-12 / 448)
    rc, rs, _ = oracle.norm_fp8(x[5:], w)
    _check_codes(torch.from_numpy(y[5:]), torch.from_numpy(s[5:]), rc, rs, SCALE)


@pytest.mark.parametrize("o_dt,g_dt", [(bf16, bf16), (f32, bf16), (f32, f32), (bf16, f32)])
@pytest.mark.parametrize("rows,heads,d", [(1, 1, 64), (1, 14, 64), (3, 3, 64), (257, 14, 64), (1, 1, 128),
                                          (5, 7, 128), (300, 32, 128), (2049, 1, 64)])
def test_gated_norm(gdr, rows, heads, d, o_dt, g_dt):
    g = _gen(rows + heads + d)
    o = torch.randn(rows, heads, d, generator=g, device="cuda").to(o_dt)
    gate = (2 * torch.randn(rows, heads, d, generator=g, device="cuda")).to(g_dt)
    w = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    y, s = gdr.gated_norm_fp8(o, gate, w)
    torch.cuda.synchronize()
    assert y.shape == (rows, heads * d)
    rc, rs = oracle.gated_norm_fp8(o, gate, w)
    top = float(gate.float().abs().max())
    _check_codes(y, s, rc, rs, SCALE + (4 + 2.4 * top) * U, "gated norm")


def test_gated_norm_far_gates_and_zero_heads(gdr):
    """Gates far out on both sides, and heads of zeros: sigmoid is 1 or 0 there, no NaN."""
    o = torch.randn(4, 3, 64, generator=_gen(9), device="cuda")
    gate = torch.zeros(4, 3, 64, device="cuda")
    gate[0], gate[1] = 90.0, -90.0
    gate[2, :, ::2], gate[2, :, 1::2] = 3e38, -3e38
    o[3, 1] = 0
    w = torch.ones(64, device="cuda")
    y, s = gdr.gated_norm_fp8(o, gate, w)
    assert torch.isfinite(s).all() and torch.isfinite(y.float()).all()
    rc, rs = oracle.gated_norm_fp8(o, gate, w)
    _check_codes(y[[0, 3]], s[[0, 3]], rc[[0, 3]], rs[[0, 3]], SCALE + (4 + 2.4 * 90) * U)
    assert not _np(y)[1].any()                   # e^-90 is far below the scale's floor
    assert not _np(y)[2, 1::2].any() and _np(y)[2, ::2].any()
    assert not _np(y)[3, 64:128].any()


@pytest.mark.parametrize("dt", [bf16, f32])
@pytest.mark.parametrize("n,k", [(1, 16), (14, 896), (127, 128), (128, 144), (129, 16), (300, 1040), (3598, 896)])
def test_quantize_weight(gdr, n, k, dt):
    w = (0.05 * torch.randn(n, k, generator=_gen(n + k), device="cuda")).to(dt)
    c, s = gdr.quantize_weight_fp8(w)
    torch.cuda.synchronize()
    rc, rs = oracle.quantize_weight_fp8(w)
    _check_codes(c, s, rc, rs, 3 * U, "weights")


@pytest.mark.parametrize("dt", [bf16, f32])
@pytest.mark.parametrize("n,k", [(127, 400), (1000, 896)])
def test_quantize_weight_ties_go_to_the_even_code(gdr, n, k, dt):
    """Multiples of 1/4 under a largest value of 448 times a power of two: every
    quotient is exact, and many lie halfway between two codes."""
    g = _gen(n + k)
    w = torch.randint(-1791, 1792, (n, k), generator=g, device="cuda").float() / 4
    if dt == bf16:                             # 8 significant bits, one more than a tie needs
        w = w.to(bf16).float()
    w[::128, ::128] = 448.0
    power = torch.exp2(torch.randint(-9, 3, (-(-n // 128), -(-k // 128)), generator=g, device="cuda").float())
    w = w * power.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    c, s = gdr.quantize_weight_fp8(w.to(dt))
    torch.cuda.synchronize()
    assert torch.equal(s, power)
    rc, _ = oracle.quantize_weight_fp8(w)
    assert np.array_equal(_np(c), oracle.e4m3(rc))
    # any scale: the code of the quotient as fp32 rounds it
    w = (0.03 * torch.randn(n, k, generator=g, device="cuda")).to(dt)
    c, s = gdr.quantize_weight_fp8(w)
    q = w.float() / s.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    assert np.array_equal(_np(c), oracle.e4m3(q))


def test_quantize_weight_special_blocks(gdr):
    w = torch.randn(256, 256, generator=_gen(11), device="cuda")
    w[:128, :128] = 0
    w[3, 200] = float("nan")
    w[200, 5] = float("-inf")
    c, s = (_np(t) for t in gdr.quantize_weight_fp8(w))
    assert s[0, 0] == np.float32(1e-12) / np.float32(448) and not c[:128, :128].any()
    assert np.isnan(s[0, 1]) and np.isnan(c[:128, 128:]).all()
    assert np.isinf(s[1, 0]) and np.isnan(c[200, 5])
    rest = c[128:, :128].copy()
    rest[72, 5] = 0
    assert not rest.any()
    rc, rs = oracle.quantize_weight_fp8(w[128:, 128:])
    assert np.allclose(s[1:, 1:], rs, rtol=3 * U)


# --- linear ----------------------------------------------------------------------------------

def _codes(g, rows, width, lo=-1.0):
    """Codes of normal values, and scales around 1 / 64 that differ by group."""
    c = (lo + 60 * torch.randn(rows, width, generator=g, device="cuda")).clamp(-448, 448).to(e4m3)
    s = (0.5 + torch.rand(rows, -(-width // 128), generator=g, device="cuda")) / 64
    return c, s


def _operands(seed, rows, n, k):
    g = _gen(seed)
    x, xs = _codes(g, rows, k)
    w, _ = _codes(g, n, k, lo=1.0)
    ws = (0.5 + torch.rand(-(-n // 128), -(-k // 128), generator=g, device="cuda")) / 64
    return x, xs, w, ws


def _check_linear(outs, ops, cols, k):
    y, size = oracle.linear_fp8(*ops)
    at = 0
    for t, c in zip(outs, cols):
        r, z = y[:, at:at + c], size[:, at:at + c]
        tol = (k + -(-k // 128) + 8) * 2 * U * z
        if t.dtype == bf16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(r)
        bad = np.abs(_np(t) - r) > tol
        assert t.shape == r.shape and not bad.any(), f"columns {at}..{at + c}: {bad.sum()} of {bad.size} out of bound"
        at += c


ROWS = [1, 2, 15, 16, 17, 36, 64, 65, 127, 128, 129, 256, 257, 511, 1000]


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("n,k", [(896, 896), (3598, 896), (130, 144)])
def test_linear_rows(gdr, rows, n, k):
    ops = _operands(rows + n, rows, n, k)
    for dt in (bf16, f32):
        y = gdr.linear_fp8(*ops, out_dtype=dt)
        torch.cuda.synchronize()
        _check_linear([y], ops, [n], k)
    gdr.linear_fp8_status()


@pytest.mark.parametrize("rows", [1, 40, 300, 2100])
@pytest.mark.parametrize("n", [1, 2, 14, 100, 127, 128, 129, 255, 256, 257, 640])
@pytest.mark.parametrize("k", [16, 128, 272, 1040])
def test_linear_columns_and_depths(gdr, rows, n, k):
    ops = _operands(rows + 7 * n + k, rows, n, k)
    y = gdr.linear_fp8(*ops, out_dtype=f32)
    torch.cuda.synchronize()
    _check_linear([y], ops, [n], k)


@pytest.mark.parametrize("rows", [700, 2100, 20000])
@pytest.mark.parametrize("n", [8, 132, 200, 264, 520, 776])
@pytest.mark.parametrize("dt", [bf16, f32])
def test_linear_last_tile_partly_empty(gdr, rows, n, dt):
    """Rows that TMA can store, and a last tile with less than half of its columns."""
    ops = _operands(rows + n, rows, n, 144)
    buf = torch.full((rows * n + 2 * 128,), 77.0, dtype=dt, device="cuda")
    out = buf[128:128 + rows * n].view(rows, n)
    gdr.linear_fp8(*ops, out_dtype=dt, out=out)
    torch.cuda.synchronize()
    at = torch.cat([torch.arange(0, 40), torch.arange(rows - 40, rows)]).cuda()
    _check_linear([out[at]], (ops[0][at], ops[1][at], *ops[2:]), [n], 144)
    assert (buf[:128] == 77).all() and (buf[-128:] == 77).all()


@pytest.mark.parametrize("rows", [1, 20, 200, 1030])
@pytest.mark.parametrize("cols,kinds", [((896, 896, 896, 896, 14), "bbbff"), ((130, 3, 1), "bfb"), ((1, 255), "fb"),
                                        ((64,) * 8, "bfbfbfbf"), ((256, 257, 127), "fbf")])
def test_linear_splits(gdr, rows, cols, kinds):
    n, k = sum(cols), 400
    ops = _operands(rows + n, rows, n, k)
    dts = [bf16 if c == "b" else f32 for c in kinds]
    outs = gdr.linear_fp8(*ops, splits=cols, out_dtype=dts)
    torch.cuda.synchronize()
    assert [t.dtype for t in outs] == dts
    _check_linear(outs, ops, cols, k)


@pytest.mark.parametrize("rows,n,k", [(1, 512, 4096), (33, 300, 4096), (128, 256, 8192), (700, 512, 4096), (4096, 1024, 1024)])
def test_linear_is_exact_where_fp32_is(gdr, rows, n, k):
    """Small whole codes and scales that are powers of two: every partial sum is an
    fp32 value, so each output must be equal, whatever the order of the sums."""
    g = _gen(rows + n + k)
    x = torch.randint(-4, 5, (rows, k), generator=g, device="cuda").float().to(e4m3)
    w = torch.randint(-4, 5, (n, k), generator=g, device="cuda").float().to(e4m3)
    xs = torch.exp2(torch.randint(-2, 2, (rows, k // 128), generator=g, device="cuda").float())
    ws = torch.exp2(torch.randint(-2, 2, (-(-n // 128), k // 128), generator=g, device="cuda").float())
    y = gdr.linear_fp8(x, xs, w, ws, out_dtype=f32)
    a = x.double() * xs.double().repeat_interleave(128, 1)
    b = w.double() * ws.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
    assert torch.equal(y.double(), a @ b.T)


@pytest.mark.parametrize("rows", [3, 130, 1100])
def test_linear_writes_its_outputs_only(gdr, rows):
    """Outputs in the middle of larger buffers, at element alignment: what lies around them stays."""
    cols, k = (129, 70, 57), 272
    ops = _operands(rows, rows, sum(cols), k)
    dts = (bf16, f32, bf16)
    ref = gdr.linear_fp8(*ops, splits=cols, out_dtype=dts)
    bufs = [torch.full((rows * c + 2 * 131,), 77.0, dtype=t, device="cuda") for c, t in zip(cols, dts)]
    outs = [b[131:131 + rows * c].view(rows, c) for b, c in zip(bufs, cols)]
    got = gdr.linear_fp8(*ops, splits=cols, out_dtype=dts, out=outs)
    for g_, r, b in zip(got, ref, bufs):
        assert torch.equal(g_, r)
        assert (b[:131] == 77).all() and (b[-131:] == 77).all()


@pytest.mark.parametrize("rows", [2, 90, 600])
def test_linear_nan_and_inf_stay_in_their_rows(gdr, rows):
    ops = _operands(rows + 3, rows, 300, 384)
    x, xs, w, ws = ops
    clean = gdr.linear_fp8(*ops, out_dtype=f32)
    x2 = x.view(torch.uint8).clone()
    x2[0, 130] = 0x7F                               # NaN code
    xs2 = xs.clone()
    xs2[1, 2] = float("inf")
    y = gdr.linear_fp8(x2.view(e4m3), xs2, w, ws, out_dtype=f32)
    assert torch.isnan(y[0]).all() and not torch.isfinite(y[1]).any()
    assert torch.equal(y[2:], clean[2:])


def test_empty_calls(gdr):
    w, ws = gdr.quantize_weight_fp8(torch.randn(40, 64, device="cuda"))
    y = gdr.linear_fp8(torch.zeros(0, 64, dtype=e4m3, device="cuda"), torch.zeros(0, 1, device="cuda"), w, ws)
    assert y.shape == (0, 40)
    y, s = gdr.norm_fp8(torch.zeros(0, 64, dtype=bf16, device="cuda"), torch.ones(64, device="cuda"))
    assert y.shape == (0, 64) and s.shape == (0, 1)
    y, s = gdr.gated_norm_fp8(torch.zeros(0, 2, 64, device="cuda"), torch.zeros(0, 2, 64, device="cuda"),
                              torch.ones(64, device="cuda"))
    assert y.shape == (0, 128) and s.shape == (0, 1)
    c, s = gdr.quantize_weight_fp8(torch.zeros(0, 64, device="cuda"))
    assert c.shape == (0, 64) and s.shape == (0, 1)


def test_misaligned_tensors_are_refused(gdr):
    buf = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    x = buf[8:8 + 128].view(e4m3).view(1, 128)
    one = torch.ones(1, 1, device="cuda")
    with pytest.raises(ValueError, match="16-byte aligned"):
        gdr.linear_fp8(x, one, torch.zeros(1, 128, dtype=e4m3, device="cuda"), one)
    xb = buf[2:2 + 256].view(bf16).view(1, 128)
    with pytest.raises(ValueError, match="16-byte aligned"):
        gdr.norm_fp8(xb, torch.ones(128, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        gdr.norm_fp8(torch.zeros(4, 256, device="cuda")[:, :128], torch.ones(128, device="cuda"))


def test_same_bits_on_every_run_and_stream(gdr):
    ops = _operands(77, 50, 1000, 2048)
    ref = gdr.linear_fp8(*ops, out_dtype=f32).clone()
    big = _operands(78, 1500, 1000, 1024)
    ref_big = gdr.linear_fp8(*big, out_dtype=f32).clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(10):
        with torch.cuda.stream(s1):
            outs.append((gdr.linear_fp8(*ops, out_dtype=f32), ref))
        with torch.cuda.stream(s2):
            outs.append((gdr.linear_fp8(*big, out_dtype=f32), ref_big))
    torch.cuda.synchronize()
    for y, r in outs:
        assert torch.equal(y, r)
    gdr.linear_fp8_status()


def test_captured_chain_replays_on_new_inputs(gdr):
    """norm -> linear with splits -> gated norm -> linear in one CUDA graph."""
    g = _gen(21)
    rows, H, d = 20, 4, 64
    c = H * d
    x = torch.randn(rows, c, generator=g, device="cuda").to(bf16)
    r = torch.randn(rows, c, generator=g, device="cuda").to(bf16)
    nw, hw = torch.ones(c, device="cuda"), torch.ones(d, device="cuda")
    w1 = gdr.quantize_weight_fp8(torch.randn(2 * c, c, generator=g, device="cuda") / c ** 0.5)
    w2 = gdr.quantize_weight_fp8(torch.randn(c, c, generator=g, device="cuda") / c ** 0.5)
    norm = gdr.PreparedNormFp8(x, nw, residual=r)
    up = gdr.PreparedLinearFp8(*norm.outputs[:2], *w1, splits=(c, c))
    gated = gdr.PreparedGatedNormFp8(up.outputs[0].view(rows, H, d), up.outputs[1].view(rows, H, d), hw)
    down = gdr.PreparedLinearFp8(*gated.outputs, *w2)

    def chain():
        norm.run()
        up.run()
        gated.run()
        return down.run()

    chain()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for seed in (1, 2):
        x.copy_(torch.randn(rows, c, generator=_gen(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*norm.outputs, *up.outputs, *gated.outputs, down.outputs)]
        for t in (*norm.outputs, *up.outputs, *gated.outputs, down.outputs):
            t.zero_()
        chain()
        for a, b in zip(got, (*norm.outputs, *up.outputs, *gated.outputs, down.outputs)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def _layer(seed, H, d, scalar):
    """Stacked projections, norms and conv taps of one mixer layer."""
    g = torch.Generator().manual_seed(seed)
    c = H * d
    gates = H if scalar else c
    n = 3 * c + gates + H
    return dict(g=g, cols=(c, c, c, gates, H), w_in=torch.randn(n, c, generator=g) / c ** 0.5,
                w_out=torch.randn(c, c, generator=g) / c ** 0.5, norm=1 + 0.1 * torch.randn(c, generator=g),
                head_norm=1 + 0.1 * torch.randn(d, generator=g),
                taps=[torch.tensor([0, 0, 0, 1.0]) + 0.1 * torch.randn(c, 4, generator=g) for _ in range(3)],
                bias=torch.full((H,) if scalar else (H, d), 5.0))


@pytest.mark.parametrize("H,d,scalar", [(3, 64, False), (2, 128, True)])
def test_mixer_layer_from_residual_stream_to_output(gdr, H, d, scalar):
    """A whole layer on two packed sequences: norm, stacked projections, the prefill
    from raw projections, gated norm, output projection; each step against the
    oracle on the bits that the step before it wrote."""
    L = _layer(5, H, d, scalar)
    c, lengths = H * d, [70, 131]
    T = sum(lengths)
    cu = torch.tensor([0, 70, 201], dtype=torch.int32)
    x = torch.randn(T, c, generator=L["g"]).to(bf16).cuda()
    r = torch.randn(T, c, generator=L["g"]).to(bf16).cuda()
    gate = torch.randn(T, H, d, generator=L["g"]).to(bf16).cuda()
    w_in, w_out = gdr.quantize_weight_fp8(L["w_in"].cuda()), gdr.quantize_weight_fp8(L["w_out"].cuda())
    y, ys, h = gdr.norm_fp8(x, L["norm"].cuda(), residual=r)
    raw = gdr.linear_fp8(y, ys, *w_in, splits=L["cols"], out_dtype=(bf16, bf16, bf16, f32, f32))
    xq, xk, xv = (t.view(T, H, d) for t in raw[:3])
    a_raw = raw[3] if scalar else raw[3].view(T, H, d)
    taps, bias = [t.cuda() for t in L["taps"]], L["bias"].cuda()
    o, _, _ = gdr.prefill_from_projections(xq, xk, xv, *taps, raw[4], a_raw, bias, cu.cuda(), scalar_decay=scalar)
    z, zs = gdr.gated_norm_fp8(o, gate, L["head_norm"].cuda())
    out = gdr.linear_fp8(z, zs, *w_out, out_dtype=f32)
    torch.cuda.synchronize()
    gdr.linear_fp8_status()

    _check_codes(y, ys, *oracle.norm_fp8(x, L["norm"], r)[:2], SCALE)
    _check_linear(raw, (y, ys, *w_in), L["cols"], c)
    act = oracle.preprocess(xq, xk, xv, *L["taps"], raw[4], a_raw, L["bias"], cu, scalar_decay=scalar)
    cast = [torch.from_numpy(act[k]).to(bf16) for k in "qkv"]
    ref = oracle.prefill(*cast, act["beta"], act["log_a"], cu, scalar_decay=scalar)["o"]
    assert np.abs(_np(o) - ref).max() <= 2e-2 * np.abs(ref).max()          # the prefill's bound
    top = float(gate.float().abs().max())
    _check_codes(z, zs, *oracle.gated_norm_fp8(o, gate, L["head_norm"]), SCALE + (4 + 2.4 * top) * U)
    _check_linear([out], (z, zs, *w_out), (c,), c)


def test_decode_layer_on_fp32_outputs(gdr):
    """The same chain for one token of each of 9 sequences around ``decode_step``."""
    H, d, B = 3, 64, 9
    L = _layer(6, H, d, False)
    c = H * d
    x = torch.randn(B, c, generator=L["g"]).to(bf16).cuda()
    gate = torch.randn(B, H, d, generator=L["g"]).to(bf16).cuda()
    state = (0.1 * torch.randn(B, H, d, d, generator=L["g"])).cuda()
    w_in, w_out = gdr.quantize_weight_fp8(L["w_in"].cuda()), gdr.quantize_weight_fp8(L["w_out"].cuda())
    y, ys = gdr.norm_fp8(x, L["norm"].cuda())
    raw = gdr.linear_fp8(y, ys, *w_in, splits=L["cols"], out_dtype=(bf16, bf16, bf16, f32, f32))
    act = gdr.preprocess(*(t.view(B, H, d) for t in raw[:3]), *(t.cuda() for t in L["taps"]), raw[4],
                         raw[3].view(B, H, d), L["bias"].cuda(), torch.arange(B + 1, dtype=torch.int32, device="cuda"))
    before = state.clone()
    o = gdr.decode_step(state, act["q"], act["k"], act["v"], act["beta"], act["log_a"])
    z, zs = gdr.gated_norm_fp8(o, gate, L["head_norm"].cuda())
    out = gdr.linear_fp8(z, zs, *w_out)
    torch.cuda.synchronize()
    _check_linear(raw, (y, ys, *w_in), L["cols"], c)
    _, ro = oracle.decode_step(before.cpu(), *(act[k].cpu() for k in ("q", "k", "v", "beta", "log_a")))
    assert np.abs(_np(o) - ro).max() <= 1e-4 * np.abs(ro).max()            # the decode step's bound
    _check_codes(z, zs, *oracle.gated_norm_fp8(o, gate, L["head_norm"]),
                 SCALE + (4 + 2.4 * float(gate.float().abs().max())) * U)
    _check_linear([out], (z, zs, *w_out), (c,), c)


# --- further calls -----------------------------------------------------------------------------

def test_offsets_past_32_bits(gdr):
    """More than 2^32 elements: the last rows are right, and so are rows in between."""
    g = _gen(41)
    rows, width = 131200, 32768                            # 4.3e9 elements
    x = torch.zeros(rows, width, dtype=bf16, device="cuda")
    at = torch.tensor([0, 65535, 65536, 131071, 131072, rows - 1], device="cuda")
    x[at] = torch.randn(at.numel(), width, generator=g, device="cuda").to(bf16)
    w = 1 + 0.1 * torch.randn(width, generator=g, device="cuda")
    y, s = gdr.norm_fp8(x, w)
    torch.cuda.synchronize()
    rc, rs, _ = oracle.norm_fp8(x[at], w)
    _check_codes(y[at], s[at], rc, rs, SCALE, "norm")
    assert not y[1].float().any() and not y[rows - 2].float().any()
    del y, s
    gate = torch.zeros(rows, 256, 128, dtype=bf16, device="cuda")
    y, s = gdr.gated_norm_fp8(x.view(rows, 256, 128), gate, w[:128].contiguous())
    torch.cuda.synchronize()
    rc, rs = oracle.gated_norm_fp8(x.view(rows, 256, 128)[at], gate[at], w[:128])
    _check_codes(y[at], s[at], rc, rs, SCALE + 4 * U, "gated norm")
    del y, s, gate
    c, s = gdr.quantize_weight_fp8(x)
    torch.cuda.synchronize()
    last = (rows - 1) // 128 * 128
    rc, rs = oracle.quantize_weight_fp8(x[last:])
    _check_codes(c[last:], s[last // 128:], rc, rs, 3 * U, "weights")
    del x, c, s
    rows, n, k = 66000, 66000, 16                          # 4.36e9 outputs
    ops = _operands(42, rows, n, k)
    out = gdr.linear_fp8(*ops)
    torch.cuda.synchronize()
    for rs_ in (slice(0, 3), slice(65534, 65540), slice(rows - 3, rows)):
        sub = (ops[0][rs_], ops[1][rs_], ops[2], ops[3])
        _check_linear([out[rs_]], sub, [n], k)


def test_prepared_calls_follow_stream_and_buffers(gdr):
    """run() on another stream, and again after its inputs were written anew."""
    g = _gen(43)
    x = torch.randn(33, 512, generator=g, device="cuda").to(bf16)
    w = torch.ones(512, device="cuda")
    wq = gdr.quantize_weight_fp8(torch.randn(200, 512, generator=g, device="cuda"))
    norm = gdr.PreparedNormFp8(x, w)
    lin = gdr.PreparedLinearFp8(*norm.outputs, *wq, out_dtype=f32)
    side = torch.cuda.Stream()
    for i in range(3):
        x.copy_(torch.randn(33, 512, generator=g, device="cuda"))
        side.wait_stream(torch.cuda.current_stream())
        norm.run(stream=side)
        assert lin.run(stream=side) is lin.outputs
        torch.cuda.current_stream().wait_stream(side)
        ref = gdr.linear_fp8(*gdr.norm_fp8(x, w), *wq, out_dtype=f32)
        assert torch.equal(lin.outputs, ref)


def test_two_graphs_of_the_same_calls_at_once(gdr):
    """Nothing is shared between calls: two captured graphs replayed on two streams."""
    cases = [_operands(51, 40, 600, 2048), _operands(52, 900, 600, 1024)]
    refs = [gdr.linear_fp8(*o, out_dtype=f32).clone() for o in cases]
    torch.cuda.synchronize()
    graphs = []
    for o in cases:
        plan = gdr.PreparedLinearFp8(*o, out_dtype=f32)
        plan.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                plan.run()
        graphs.append((graph, plan, torch.cuda.Stream()))
    for graph, plan, st in graphs:
        plan.outputs.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, plan, st in graphs:
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for (graph, plan, st), r in zip(graphs, refs):
        assert torch.equal(plan.outputs, r)
    gdr.linear_fp8_status()


def test_products_beside_a_prefill_on_another_stream(gdr):
    """The product's kernels and the prefill's hold tensor memory on the same SMs."""
    import workloads as wl
    w = wl.shrink(wl.VARLEN, n_heads=4, d_k=64, d_v=64, lengths=(700, 300), init_std=0.1, snap_interval=0)
    d = {k: (v.cuda() if torch.is_tensor(v) else v) for k, v in wl.make_prefill_inputs(w).items()}
    pre = lambda: gdr.prefill(d["q"], d["k"], d["v"], d["beta"], d["log_a"], d["cu_seqlens"],
                              init_state=d["init_state"], cu_seqlens_host=d["cu_seqlens"].cpu())[0]
    cases = [_operands(61, 30, 2000, 2048), _operands(62, 300, 2000, 1024), _operands(63, 2000, 2000, 512)]
    refs = [gdr.linear_fp8(*o) for o in cases]
    o_ref = pre()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs, os_ = [], []
    for _ in range(8):
        with torch.cuda.stream(streams[3]):
            os_.append(pre())
        for o, r, st in zip(cases, refs, streams):
            with torch.cuda.stream(st):
                outs.append((gdr.linear_fp8(*o), r))
    torch.cuda.synchronize()
    assert all(torch.equal(y, r) for y, r in outs)
    assert all(torch.equal(o, o_ref) for o in os_)
    gdr.linear_fp8_status()


@pytest.mark.parametrize("cols,kinds", [((3598,), "b"), ((1001,), "b"), ((1001,), "f"), ((2050,), "f"), ((896, 14, 1030), "bfb"),
                                        ((129, 70, 57, 1000), "bfbf"), ((3, 14, 777, 5, 300, 1, 131, 260), "bbfbbfbf")])
@pytest.mark.parametrize("rows", [515, 4099])
def test_linear_rows_at_any_alignment(gdr, rows, cols, kinds):
    """Products for many tokens whose output rows start at any element, in the middle
    of larger buffers.  Each output is its sum rounded once, so it is equal to one
    wide fp32 product (or that, rounded), and what lies around it stays."""
    n, k = sum(cols), 272
    wide = -(-n // 8) * 8 + 8                          # the reference's rows are aligned
    x, xs, w, ws = _operands(rows + n, rows, wide, k)
    ref = gdr.linear_fp8(x, xs, w, ws, out_dtype=f32)
    at = torch.cat([torch.arange(0, 3), torch.arange(rows - 3, rows)]).cuda()
    _check_linear([ref[at]], (x[at], xs[at], w, ws), [wide], k)
    dts = [bf16 if c == "b" else f32 for c in kinds]
    ws_n = ws[:-(-n // 128)].contiguous()
    for lead in (128, 131, 134, 137):
        bufs = [torch.full((rows * c + lead + 128,), 77.0, dtype=t, device="cuda") for c, t in zip(cols, dts)]
        outs = [b[lead:lead + rows * c].view(rows, c) for b, c in zip(bufs, cols)]
        gdr.linear_fp8(x, xs, w[:n].contiguous(), ws_n, splits=cols, out_dtype=dts, out=outs)
        for o, b, r, t in zip(outs, bufs, ref[:, :n].split(cols, 1), dts):
            assert torch.equal(o, r.to(t))
            assert (b[:lead] == 77).all() and (b[-128:] == 77).all()
    gdr.linear_fp8_status()


@pytest.mark.parametrize("rows", [297, 300, 303, 1001, 40001])
@pytest.mark.parametrize("width", [16, 64, 112, 128, 144, 240, 256, 272])
@pytest.mark.parametrize("dt,residual", [(bf16, True), (f32, False), (f32, True)])
def test_norm_many_narrow_rows(gdr, rows, width, dt, residual):
    """More than one row to a warp, and a last warp that is not full."""
    _check_norm(gdr, rows, width, dt, residual, seed=2)
