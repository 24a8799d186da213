"""Comparisons of 8-bit results with the fp64 oracle that a NaN cannot pass: each
asserts that every element is within its bound (a NaN is within none), instead of
that none is outside.  The bounds are those derived in test_fp8_gpu.py."""
import numpy as np
import torch

U = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


def as_np(t):
    return t.double().cpu().numpy() if torch.is_tensor(t) else np.asarray(t, dtype=np.float64)


def assert_within(got, ref, tol, what):
    got, ref = as_np(got), as_np(ref)
    assert got.shape == ref.shape, f"{what}: shape {got.shape}, expected {ref.shape}"
    ok = np.abs(got - ref) <= tol
    assert ok.all(), f"{what}: {(~ok).sum()} of {ok.size} out of bound, {np.isnan(got).sum()} NaN"


def check_codes(codes, scale, ref_codes, ref_scale, tol, what=""):
    """Scales within `tol`; each code within half a step of e4m3 of the oracle's
    quotient, whose own error is under twice the scale's."""
    assert_within(scale, ref_scale, tol * ref_scale, f"{what} scale")
    t = np.abs(ref_codes) * (1 + 2 * np.max(tol))
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(t, 1e-30))), -6.0) - 3)
    assert_within(codes, ref_codes, step / 2 + 2 * np.max(tol) * np.abs(ref_codes), f"{what} codes")


def check_linear(outs, ref, cols, k):
    """`ref`: the oracle's (product, sum of its terms' sizes)."""
    y, size = ref
    at = 0
    for t, c in zip(outs, cols):
        r = y[:, at:at + c]
        tol = (k + -(-k // 128) + 8) * 2 * U * size[:, at:at + c]
        if t.dtype == torch.bfloat16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(r)
        assert_within(t, r, tol, f"columns {at}..{at + c}")
        at += c


def nan_filled(*shape, dtype, device="cuda"):
    """A tensor of NaN: what a kernel leaves unwritten fails every check."""
    if dtype == E4M3:
        return torch.full(shape, 0x7F, dtype=torch.uint8, device=device).view(E4M3)
    return torch.full(shape, float("nan"), dtype=dtype, device=device)
