"""The comparisons of fp8_checks.py refuse one NaN, one unwritten element and one
element out of bound, and accept results within their bounds."""
import numpy as np
import pytest
import torch

import oracle
from fp8_checks import check_codes, check_linear, nan_filled

bf16, f32, e4m3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _codes_case():
    y = np.random.default_rng(1).standard_normal((5, 272))
    codes, scale = oracle._scaled_rows(y)
    return torch.from_numpy(oracle.e4m3(codes)).to(e4m3), torch.from_numpy(scale).float(), codes, scale


def test_codes():
    c, s, rc, rs = _codes_case()
    check_codes(c, s, rc, rs, 1e-6)
    for at in ((0, 0), (4, 271)):
        bad = c.view(torch.uint8).clone()
        bad[at] = 0x7F
        with pytest.raises(AssertionError, match="1 NaN"):
            check_codes(bad.view(e4m3), s, rc, rs, 1e-6)
        off = c.float()
        off[at] += 64
        with pytest.raises(AssertionError, match="out of bound"):
            check_codes(off, s, rc, rs, 1e-6)
    bad = s.clone()
    bad[2, 1] = float("nan")
    with pytest.raises(AssertionError, match="scale: 1 of"):
        check_codes(c, bad, rc, rs, 1e-6)
    with pytest.raises(AssertionError, match="shape"):
        check_codes(c[:4], s, rc, rs, 1e-6)
    with pytest.raises(AssertionError):
        check_codes(nan_filled(5, 272, dtype=e4m3, device="cpu"), s, rc, rs, 1e-6)


@pytest.mark.parametrize("dt", [bf16, f32])
def test_linear(dt):
    r = np.random.default_rng(2)
    x, w = oracle._scaled_rows(r.standard_normal((3, 160))), oracle.quantize_weight_fp8(r.standard_normal((130, 160)))
    ref = oracle.linear_fp8(*x, *w)
    outs = [t.to(dt) for t in torch.from_numpy(ref[0]).split([100, 30], 1)]
    check_linear(outs, ref, (100, 30), 160)
    for value in (float("nan"), float("inf"), 1e3):
        bad = [t.clone() for t in outs]
        bad[1][2, 29] = value
        with pytest.raises(AssertionError, match="columns 100..130: 1 of"):
            check_linear(bad, ref, (100, 30), 160)
    with pytest.raises(AssertionError, match="300 NaN"):
        check_linear([nan_filled(3, 100, dtype=dt, device="cpu"), outs[1]], ref, (100, 30), 160)
