"""What is measured of the 8-bit projections around the gated delta-rule mixer.

A hybrid model's mixer layer reads the residual stream through an RMSNorm and
one matrix product (q, k, v, decay and write-strength projections), and writes
back through a gated per-head RMSNorm and another matrix product.  With 8-bit
weights (e4m3, one fp32 scale for each 128 x 128 block) and 8-bit activations
(e4m3, one fp32 scale for each token and 128 channels) the operators are

  norm      h = x + residual;  y = h / sqrt(mean h^2 + eps) * w, given as codes and scales
  gated     y = o / sqrt(mean o^2 + eps) * w * sigmoid(gate) per head, as codes and scales
  linear    y = (codes * scales) (codes * scales)^T, cut into column ranges of their own types
  quantize  a weight matrix as codes and block scales (when a model is loaded)

A group's scale is max(max |y|, 1e-12) / 448 and its codes are y / scale rounded
to e4m3.  A width that is no multiple of 128 leaves a shorter last group.

`run` computes them in elementary torch operations, or, where `own` is set,
through the package's entry points.
"""
import math

import torch

own = False

GROUP = 128
EPS = 1e-6
E4M3_MAX = 448.0
FLOOR = 1e-12
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
TYPES = {"bf16": BF16, "f32": F32}


def listed():
    return [
        # one decoded token on the 14-head, d 64 graft layer (hidden width 896)
        {"name": "norm_token_896", "op": "norm", "rows": 1, "width": 896, "type": "bf16", "residual": True},
        # the graft layer's 8192-token prompt
        {"name": "norm_graft_prompt", "op": "norm", "rows": 8192, "width": 896, "type": "bf16", "residual": True},
        # the 65536-token prompt of the 16-head, d 128 model (hidden width 2048)
        {"name": "norm_long_prompt", "op": "norm", "rows": 65536, "width": 2048, "type": "bf16", "residual": True},
        # the decode batch of 256: the decode step's fp32 outputs, 14 heads of 64
        {"name": "gated_decode_256", "op": "gated", "rows": 256, "heads": 14, "d": 64, "type": "f32", "gate": "bf16"},
        # a packed prompt batch, 32 heads of 128
        {"name": "gated_prompt_32x128", "op": "gated", "rows": 16384, "heads": 32, "d": 128, "type": "bf16", "gate": "bf16"},
        # one token's q, k, v, decay and beta projections on the graft layer
        {"name": "linear_token_graft", "op": "linear", "rows": 1, "k": 896, "cols": "896b,896b,896b,896f,14f"},
        # 4 draft tokens for each of 9 sequences, output projection of the 32-head model
        {"name": "linear_draft_4096", "op": "linear", "rows": 36, "k": 4096, "cols": "4096b"},
        # the decode batch of 256 on the 32-head, d 128 model, per-channel decay
        {"name": "linear_decode_256", "op": "linear", "rows": 256, "k": 4096, "cols": "4096b,4096b,4096b,4096f,32f"},
        # the graft layer's prompt
        {"name": "linear_graft_prompt", "op": "linear", "rows": 8192, "k": 896, "cols": "896b,896b,896b,896f,14f"},
        # q, k, v of a packed prompt batch with an odd token count, scalar decay, 32 heads of 128
        {"name": "linear_prompt_4096", "op": "linear", "rows": 16381, "k": 4096, "cols": "4096b,4096b,4096b,32f,32f"},
        # loading the graft layer's and the 32-head model's stacked projections
        {"name": "quantize_graft", "op": "quantize", "n": 3598, "k": 896, "type": "bf16"},
        {"name": "quantize_16416x4096", "op": "quantize", "n": 16416, "k": 4096, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of lo .. hi."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gated", "linear", "linear", "linear", "quantize"])
    if op == "norm":
        width = 16 * _log(rng, 4, 512)
        return {"op": op, "rows": _log(rng, 1, min(65536, 65536 * 2048 // width)), "width": width,
                "type": rng.choice(["bf16", "bf16", "f32"]) if width < 4096 else "bf16",
                "residual": rng.random() < 0.75}
    if op == "gated":
        d, heads = rng.choice([64, 128]), rng.randint(1, 40)
        return {"op": op, "rows": _log(rng, 1, min(65536, 65536 * 1024 // (d * heads))), "heads": heads, "d": d,
                "type": rng.choice(["bf16", "f32"]), "gate": rng.choice(["bf16", "bf16", "f32"])}
    if op == "quantize":
        k = 16 * _log(rng, 4, 512)
        return {"op": op, "n": _log(rng, 1, min(16416, 16416 * 4096 // k)), "k": k, "type": rng.choice(["bf16", "f32"])}
    k = 16 * _log(rng, 4, 512)
    kind = rng.randrange(3)
    if kind == 0:       # a whole mixer's projections, per-channel or scalar decay
        heads, d = rng.randint(2, 32), rng.choice([64, 128])
        c = heads * d
        cols = "%db,%db,%db,%df,%df" % (c, c, c, c if rng.random() < 0.5 else heads, heads)
    elif kind == 1:     # one product, any width
        cols = "%d%s" % (_log(rng, 1, 16384), rng.choice("bf"))
    else:               # two ranges that begin anywhere
        cols = "%d%s,%d%s" % (_log(rng, 1, 4096), rng.choice("bf"), _log(rng, 1, 4096), rng.choice("bf"))
    n = sum(w for w, _ in _cols(cols))
    return {"op": op, "rows": _log(rng, 1, max(1, min(32768, 16381 * 12352 * 4096 // (n * k)))), "k": k, "cols": cols}


def _cols(text):
    """Widths and types of the output's column ranges, e.g. "896b,14f"."""
    return [(int(t[:-1]), BF16 if t[-1] == "b" else F32) for t in text.split(",")]


def _groups(n):
    return -(-n // GROUP)


# --- plain forms -----------------------------------------------------------------------------

def _plain_codes(y):
    """fp32 rows as e4m3 codes and one scale for each row and 128 columns."""
    rows, width = y.shape
    pad = _groups(width) * GROUP - width
    g = torch.nn.functional.pad(y, (0, pad)).view(rows, -1, GROUP)
    scale = g.abs().amax(-1).clamp_min(FLOOR) / E4M3_MAX
    codes = (g / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, -1)[:, :width]
    return codes.contiguous().to(E4M3), scale


def _plain_blocks(w):
    """fp32 matrix as e4m3 codes and one scale for each 128 x 128 block."""
    n, k = w.shape
    p = torch.nn.functional.pad(w, (0, _groups(k) * GROUP - k, 0, _groups(n) * GROUP - n))
    p = p.view(_groups(n), GROUP, _groups(k), GROUP)
    scale = p.abs().amax((1, 3)).clamp_min(FLOOR) / E4M3_MAX
    codes = (p / scale[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    return codes.reshape(_groups(n) * GROUP, -1)[:n, :k].contiguous().to(E4M3), scale


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    codes, scale = _plain_codes(y)
    return [codes, scale] if s["residual"] is None else [codes, scale, h.to(s["x"].dtype)]


def _plain_gated(s):
    o = s["o"].float()
    y = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS) * s["weight"] * torch.sigmoid(s["gate"].float())
    return list(_plain_codes(y.flatten(1)))


def _plain_linear(s):
    n, k = s["w"].shape
    x = s["x"].float() * s["x_scale"].repeat_interleave(GROUP, 1)[:, :k]
    w = s["w"].float() * s["w_scale"].repeat_interleave(GROUP, 0)[:n].repeat_interleave(GROUP, 1)[:, :k]
    y = x @ w.T
    return [c.to(t) for c, (_, t) in zip(y.split([w for w, _ in s["cols"]], 1), s["cols"])]


# --- the measured path -----------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32)


def _activations(g, rows, width):
    """A residual stream: unit-size values, a few channels an order of magnitude above the rest."""
    loud = 1 + 20 * (torch.rand(width, generator=g, device="cuda") < 0.01)
    return _normal(g, rows, width) * loud


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op == "norm":
        dt = TYPES[case["type"]]
        s["x"] = _normal(g, case["rows"], case["width"]).to(dt)
        s["residual"] = _activations(g, case["rows"], case["width"]).to(dt) if case["residual"] else None
        s["weight"] = 1 + 0.1 * _normal(g, case["width"])
    elif op == "gated":
        s["o"] = (0.3 * _normal(g, case["rows"], case["heads"], case["d"])).to(TYPES[case["type"]])
        s["gate"] = _normal(g, case["rows"], case["heads"], case["d"]).to(TYPES[case["gate"]])
        s["weight"] = 1 + 0.1 * _normal(g, case["d"])
    elif op == "linear":
        s["cols"] = _cols(case["cols"])
        n, k = sum(w for w, _ in s["cols"]), case["k"]
        s["x"], s["x_scale"] = _plain_codes(_activations(g, case["rows"], k))
        s["w"], s["w_scale"] = _plain_blocks(_normal(g, n, k) * (0.02 + 0.02 * torch.rand(n, 1, generator=g, device="cuda")))
    else:
        s["w"] = (0.03 * _normal(g, case["n"], case["k"])).to(TYPES[case["type"]])
    if own:             # the argument block that a serving loop builds once over its own buffers
        import gated_delta_rule_150_b200 as gdr
        s["gdr"] = gdr
        if op == "norm":
            s["plan"] = gdr.PreparedNormFp8(s["x"], s["weight"], residual=s["residual"], norm_eps=EPS)
        elif op == "gated":
            s["plan"] = gdr.PreparedGatedNormFp8(s["o"], s["gate"], s["weight"], norm_eps=EPS)
        elif op == "linear":
            s["plan"] = gdr.PreparedLinearFp8(s["x"], s["x_scale"], s["w"], s["w_scale"],
                                              splits=[w for w, _ in s["cols"]], out_dtype=[t for _, t in s["cols"]])
    return s


def run(s):
    op = s["op"]
    if own:
        if op == "quantize":
            return list(s["gdr"].quantize_weight_fp8(s["w"]))
        return s["plan"].run()
    if op == "norm":
        return _plain_norm(s)
    if op == "gated":
        return _plain_gated(s)
    if op == "linear":
        return _plain_linear(s)
    return list(_plain_blocks(s["w"].float()))


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "norm":
        n, e = case["rows"] * case["width"], size[case["type"]]
        return {"bytes": n * e * (3 if case["residual"] else 1) + n + 4 * case["rows"] * _groups(case["width"]) + 4 * case["width"],
                "flops": 7 * n}
    if op == "gated":
        n = case["rows"] * case["heads"] * case["d"]
        return {"bytes": n * (size[case["type"]] + size[case["gate"]]) + n
                + 4 * case["rows"] * _groups(case["heads"] * case["d"]) + 4 * case["d"], "flops": 10 * n}
    if op == "quantize":
        n = case["n"] * case["k"]
        return {"bytes": n * size[case["type"]] + n + 4 * _groups(case["n"]) * _groups(case["k"]), "flops": 2 * n}
    rows, k, cols = case["rows"], case["k"], _cols(case["cols"])
    n = sum(w for w, _ in cols)
    out = sum(rows * w * (2 if t is BF16 else 4) for w, t in cols)
    return {"bytes": rows * k + 4 * rows * _groups(k) + n * k + 4 * _groups(n) * _groups(k) + out, "flops": 2 * rows * n * k}


# --- the definition in 64 bits ---------------------------------------------------------------

def _exact_scaled(y):
    """Rows in 64 bits: what the codes stand for before they are rounded, and the scales."""
    codes, scale = torch.empty_like(y), y.new_empty(y.shape[0], _groups(y.shape[1]))
    for j in range(scale.shape[1]):
        part = y[:, GROUP * j:GROUP * (j + 1)]
        top = torch.maximum(part.max(1).values, -part.min(1).values)
        scale[:, j] = torch.where(top < FLOOR, torch.full_like(top, FLOOR), top) / E4M3_MAX
        codes[:, GROUP * j:GROUP * (j + 1)] = part / scale[:, j:j + 1]
    return [codes, scale]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = s["residual"].double() + h
        rms = (torch.einsum("rc,rc->r", h, h) / h.shape[1] + EPS).sqrt()
        out = _exact_scaled(h / rms[:, None] * s["weight"].double())
        return out if s["residual"] is None else out + [h]
    if op == "gated":
        o, gate = s["o"].double(), s["gate"].double()
        rms = (torch.einsum("rhc,rhc->rh", o, o) / o.shape[2] + EPS).sqrt()
        y = o / rms[..., None] * s["weight"].double() / (1 + torch.exp(-gate))
        return _exact_scaled(y.reshape(y.shape[0], -1))
    if op == "quantize":
        w = s["w"].double()
        codes, scale = torch.empty_like(w), w.new_empty(_groups(w.shape[0]), _groups(w.shape[1]))
        for i in range(scale.shape[0]):
            rows = slice(GROUP * i, GROUP * (i + 1))
            for j in range(scale.shape[1]):
                part = w[rows, GROUP * j:GROUP * (j + 1)]
                scale[i, j] = torch.linalg.vector_norm(part, float("inf")).clamp_min(FLOOR) / E4M3_MAX
                codes[rows, GROUP * j:GROUP * (j + 1)] = part / scale[i, j]
        return [codes, scale]
    n, k = s["w"].shape
    y = torch.zeros(case["rows"], n, dtype=torch.float64, device="cuda")
    block = torch.arange(n, device="cuda") // GROUP
    for j in range(_groups(k)):
        at = slice(GROUP * j, GROUP * (j + 1))
        w = s["w"][:, at].double() * s["w_scale"][block, j].double()[:, None]
        y.addmm_(s["x"][:, at].double() * s["x_scale"][:, j].double()[:, None], w.T)
    return list(torch.split(y, [c for c, _ in s["cols"]], 1))
