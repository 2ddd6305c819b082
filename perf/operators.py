"""Cases of the 8-bit floating-point operators: the block quantizer
(zr_quantize_fp8), the product of block-scaled codes (zr_matmul_fp8), the
root-mean-square norm with the residual's addition and 8-bit output
(zr_rmsnorm_fp8) and its backward pass (zr_rmsnorm_backward).

Codes are e4m3 or e5m2.  A group of 128 (or a 128 x 128 block) has one scale, a
power of two held as E8M0: 2^e with the smallest e that brings the group's
largest magnitude to at most 448 (e4m3) or 57344 (e5m2).
"""
import math

import torch
import torch.nn.functional as F

own = False

GROUP = 128
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# exponent of the formats' largest value, 1.75 * 2^8 and 1.75 * 2^15
TOP = {torch.float8_e4m3fn: 8, torch.float8_e5m2: 15}
# rows of partial sums in the norm's backward workspace
PARTIALS = 512


def listed():
    return [
        # One token's activations before a projection while decoding: latency.
        {"name": "quantize_token", "op": "quantize", "rows": 1, "cols": 4096, "block_rows": 1, "both": False,
         "type": "bf16", "codes": "e4m3"},
        # The input of a down projection in a training step.
        {"name": "quantize_activations", "op": "quantize", "rows": 8192, "cols": 11008, "block_rows": 1, "both": False,
         "type": "bf16", "codes": "e4m3"},
        # A gathered weight and its transposed copy, for the forward product and the input gradient.
        {"name": "quantize_weight", "op": "quantize", "rows": 11008, "cols": 4096, "block_rows": 128, "both": True,
         "type": "bf16", "codes": "e4m3"},
        # The output gradient of a fused query/key/value projection over a ragged batch, along both axes.
        {"name": "quantize_gradient", "op": "quantize", "rows": 5003, "cols": 12288, "block_rows": 1, "both": True,
         "type": "fp16", "codes": "e5m2"},
        # One decoded token through the norm before a projection: latency.
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 4096, "y": False, "type": "bf16"},
        # The norm of a training step: the stream, the normed rows (kept for the weight gradient) and their codes.
        {"name": "norm_training", "op": "norm", "rows": 16384, "cols": 4096, "y": True, "type": "bf16"},
        # Backward of a small model's norm over a ragged batch, a width that ends inside a group.
        {"name": "norm_backward_small", "op": "norm_backward", "rows": 777, "cols": 1000, "dh": False, "type": "fp16"},
        # Backward of a training step's norm, with the gradient of the residual stream.
        {"name": "norm_backward", "op": "norm_backward", "rows": 16384, "cols": 4096, "dh": True, "type": "bf16"},
        # One decoded token times a gathered gate projection, scales per row as a flat gather leaves them.
        {"name": "matmul_token", "op": "matmul", "m": 1, "n": 11008, "k": 4096, "block_rows": 1, "type": "bf16",
         "codes": "e4m3"},
        # A ragged prompt through a down projection.
        {"name": "matmul_prompt", "op": "matmul", "m": 333, "n": 4096, "k": 11008, "block_rows": 128, "type": "bf16",
         "codes": "e4m3"},
        # The up projection of a training step.
        {"name": "matmul_forward", "op": "matmul", "m": 16384, "n": 11008, "k": 4096, "block_rows": 128, "type": "bf16",
         "codes": "e4m3"},
        # Its weight gradient over a ragged batch of tokens, both operands scaled along the tokens, as the bf16
        # contribution that the gradient reduction takes.
        {"name": "matmul_weight_gradient", "op": "matmul", "m": 11008, "n": 4096, "k": 8111, "block_rows": 1,
         "type": "bf16", "codes": "e5m2"},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "norm_backward", "matmul", "matmul"])
    kind = rng.choice(["bf16", "bf16", "fp16"])
    # widths: a model's own (whole groups) or any
    width = lambda low, high: GROUP * _spread(rng, max(1, low // GROUP), high // GROUP) if rng.random() < 0.6 \
        else _spread(rng, low, high)  # noqa: E731
    if op == "matmul" and rng.random() < 0.33:  # a weight gradient
        return {"op": op, "m": width(512, 11008), "n": width(512, 4096), "k": _spread(rng, 64, 8192), "block_rows": 1,
                "type": rng.choice(["bf16", "fp32"]), "codes": rng.choice(["e4m3", "e5m2"])}
    if op == "matmul":
        n, k = width(512, 11008), width(512, 11008)
        return {"op": op, "m": _spread(rng, 1, min(16384, 700_000_000_000 // (n * k))), "n": n, "k": k,
                "block_rows": rng.choice([1, 128, 128]), "type": kind, "codes": rng.choice(["e4m3", "e4m3", "e5m2"])}
    if op == "quantize":
        rows = _spread(rng, 1, 8192)
        return {"op": op, "rows": rows, "cols": width(128, 12288), "block_rows": rng.choice([1, 1, 128]),
                "both": rows > 1 and rng.random() < 0.5, "type": kind, "codes": rng.choice(["e4m3", "e5m2"])}
    cols = width(128, 11008)
    rows = _spread(rng, 1, min(16384, 67_000_000 // cols))
    return {"op": op, "rows": rows, "cols": cols, "y" if op == "norm" else "dh": rng.random() < 0.5, "type": kind}


def _groups(n):
    return -(-n // GROUP)


def _line(n):
    """Row length of a code matrix as a program allocates it: whole 128-byte lines."""
    return _groups(n) * GROUP


def _scale_values(bytes_):
    return bytes_.view(torch.float8_e8m0fnu).float()


def _scale_bytes(amax, codes):
    """E8M0 bytes of the groups whose largest magnitudes are `amax`."""
    amax = amax.double()
    part, exponent = torch.frexp(amax)  # amax = part * 2^exponent, 0.5 <= part < 1
    e = exponent - 1 - TOP[codes] + (part > 0.875).to(exponent.dtype)
    e = torch.where(amax == 0, torch.full_like(e, -127), e.clamp(min=-127))
    return torch.where(torch.isfinite(amax), e + 127, torch.full_like(e, 255)).to(torch.uint8)


def _quantize_plain(x, codes, block_rows):
    """(codes, scale bytes) of the rows of x (fp32), in groups of 128 along a row or blocks of 128 x 128."""
    rows, cols = x.shape
    tall = _groups(rows) * block_rows if block_rows > 1 else rows
    padded = F.pad(x, (0, _line(cols) - cols, 0, tall - rows))
    blocks = padded.view(tall // block_rows, block_rows, _groups(cols), GROUP)
    s = _scale_bytes(blocks.abs().amax(dim=(1, 3)), codes)
    inverse = _scale_values(torch.where(s == 255, s, 254 - s))
    q = (blocks * inverse[:, None, :, None]).view(tall, -1)[:rows, :cols].to(codes)
    return q, s


def _values(q, s, block_rows):
    """What codes and scales stand for, in fp32."""
    scale = _scale_values(s).repeat_interleave(GROUP, dim=1)[:, :q.shape[1]]
    if block_rows > 1:
        scale = scale.repeat_interleave(block_rows, dim=0)[:q.shape[0]]
    return q.float() * scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    op, kind = case["op"], TYPES[case["type"]]
    s = dict(case)
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        # tokens' sizes differ from one to the next, gradients' by more
        a = randn(m, k) * torch.exp(randn(m, 1) * 0.5)
        b = randn(n, k) * 0.02
        for name, x, codes, block_rows in (("a", a, CODES[case["codes"]], 1), ("b", b, CODES["e4m3"], case["block_rows"])):
            q, scale = _quantize_plain(x, codes, block_rows)
            s[name] = torch.zeros(x.shape[0], _line(k), dtype=codes, device="cuda")[:, :k]
            s[name].copy_(q)
            s[name + "_scales"] = scale.view(torch.float8_e8m0fnu)
        s["out"] = torch.empty(m, n, dtype=kind, device="cuda")
        return s
    rows, cols = case["rows"], case["cols"]
    byte = lambda r, c, t: torch.zeros(r, _line(c), dtype=t, device="cuda")[:, :c]  # noqa: E731
    scales = lambda r, c: torch.empty(r, c, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)  # noqa: E731
    if op == "quantize":
        codes = CODES[case["codes"]]
        s["src"] = (randn(rows, cols) * torch.exp(randn(rows, 1))).to(kind)
        s["q"] = byte(rows, cols, codes)
        tall = rows if case["block_rows"] == 1 else _groups(rows)
        s["scales"] = scales(tall, _groups(cols))
        if case["both"]:
            s["qt"] = byte(cols, rows, codes)
            s["scales_t"] = scales(cols if case["block_rows"] == 1 else _groups(cols), _groups(rows))
        return s
    s["weight"] = (1 + 0.1 * randn(cols)).to(kind)
    s["eps"] = 1e-5
    if op == "norm":
        s["x"], s["residual"] = randn(rows, cols).to(kind), (2 * randn(rows, cols)).to(kind)
        s["h"] = torch.empty_like(s["x"])
        s["y"] = torch.empty_like(s["x"]) if case["y"] else None
        s["rstd"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        s["q"] = byte(rows, cols, torch.float8_e4m3fn)
        s["scales"] = scales(rows, _groups(cols))
        return s
    s["h"], s["dy"] = (2 * randn(rows, cols)).to(kind), randn(rows, cols).to(kind)
    s["dh"] = randn(rows, cols).to(kind) if case["dh"] else None
    s["rstd"] = torch.rsqrt(s["h"].float().square().mean(dim=1) + s["eps"])
    s["dx"], s["dweight"] = torch.empty_like(s["h"]), torch.empty_like(s["weight"])
    s["workspace"] = torch.empty(PARTIALS, cols, dtype=torch.float32, device="cuda")
    return s


def _run_own(s):
    import zero_sharded_optimizer_zr_amd as zr
    if s["op"] == "quantize":
        zr.zr_quantize_fp8(s["src"], s["q"], s["scales"], s.get("qt"), s.get("scales_t"), block_rows=s["block_rows"])
        return {k: s[k] for k in ("q", "scales", "qt", "scales_t") if k in s}
    if s["op"] == "norm":
        zr.zr_rmsnorm_fp8(s["x"], s["weight"], y=s["y"], q=s["q"], scales=s["scales"], residual=s["residual"], h=s["h"],
                          rstd=s["rstd"], eps=s["eps"])
        return {k: s[k] for k in ("h", "y", "rstd", "q", "scales")}
    if s["op"] == "norm_backward":
        zr.zr_rmsnorm_backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"], s["dweight"], s["workspace"],
                               dh=s["dh"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    zr.zr_matmul_fp8(s["a"], s["a_scales"], s["b"], s["b_scales"], s["out"], b_block_rows=s["block_rows"])
    return {"out": s["out"]}


def _run_plain(s):
    if s["op"] == "quantize":
        codes, x = CODES[s["codes"]], s["src"].float()
        q, scale = _quantize_plain(x, codes, s["block_rows"])
        out = {"q": q, "scales": scale.view(torch.float8_e8m0fnu)}
        if s["both"]:
            qt, scale_t = _quantize_plain(x.t().contiguous(), codes, s["block_rows"])
            out.update(qt=qt, scales_t=scale_t.view(torch.float8_e8m0fnu))
        return out
    if s["op"] == "norm":
        h = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
        x = h.float()
        rstd = torch.rsqrt((x * x).mean(dim=1) + s["eps"])
        y = x * rstd[:, None] * s["weight"].float()
        q, scale = _quantize_plain(y, torch.float8_e4m3fn, 1)
        return {"h": h, "y": y.to(h.dtype) if s["y"] is not None else None, "rstd": rstd, "q": q,
                "scales": scale.view(torch.float8_e8m0fnu)}
    if s["op"] == "norm_backward":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh, g = s["h"].float() * rstd, dy * s["weight"].float()
        dx = rstd * (g - xh * (g * xh).mean(dim=1, keepdim=True))
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(s["h"].dtype), "dweight": (dy * xh).sum(dim=0).to(s["weight"].dtype)}
    a = _values(s["a"], s["a_scales"].view(torch.uint8), 1)
    b = _values(s["b"], s["b_scales"].view(torch.uint8), s["block_rows"])
    return {"out": torch.matmul(a, b.t()).to(s["out"].dtype)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, size = case["op"], 4 if case["type"] == "fp32" else 2
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        b_rows = n if case["block_rows"] == 1 else _groups(n)
        return {"bytes": m * k + n * k + (m + b_rows) * _groups(k) + m * n * size, "flops": 2 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    if op == "quantize":
        copies = 2 if case["both"] else 1
        down = _groups(rows) if case["block_rows"] > 1 else rows
        across = _groups(cols) if case["block_rows"] > 1 else cols
        scales = down * _groups(cols) + (across * _groups(rows) if case["both"] else 0)
        return {"bytes": n * size + n * copies + scales, "flops": 2 * n * copies}
    if op == "norm":
        return {"bytes": n * size * (4 if case["y"] else 3) + n + rows * _groups(cols) + 4 * rows + cols * size,
                "flops": 7 * n}
    return {"bytes": n * size * (4 if case["dh"] else 3) + 4 * rows + 2 * cols * size, "flops": 11 * n}


def _exact_codes(x, codes, block_rows):
    """Unrounded codes x / 2^e and scales 2^e of x (64 bits), block by block maxima taken by pooling."""
    rows, cols = x.shape
    tall = (block_rows, GROUP)
    amax = F.max_pool2d(x.abs()[None, None], tall, ceil_mode=True)[0, 0]
    top = 1.75 * 2.0 ** TOP[codes]
    e = torch.ceil(torch.log2(amax / top))
    e = torch.where(amax > top * torch.exp2(e), e + 1, torch.where(amax <= top * torch.exp2(e - 1), e - 1, e))
    scale = torch.exp2(e.clamp(min=-127))
    wide = scale.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(GROUP, 1)[:, :cols]
    return x / wide, scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        codes, x = CODES[case["codes"]], s["src"].double()
        q, scale = _exact_codes(x, codes, case["block_rows"])
        out = {"q": q, "scales": scale}
        if case["both"]:
            out["qt"], out["scales_t"] = _exact_codes(x.t(), codes, case["block_rows"])
        if codes == torch.float8_e5m2:  # two bits of mantissa: every code is up to an eighth from any unrounded value
            out.update({k: None for k in out if not k.startswith("scales")})
        return out
    if case["op"] == "norm":
        h = s["x"].double() + s["residual"].double()
        x = h.to(s["x"].dtype).double()  # the norm is of the stream as it is kept
        rstd = 1 / torch.sqrt(x.pow(2).sum(1) / x.shape[1] + s["eps"])
        y = torch.einsum("rc,r,c->rc", x, rstd, s["weight"].double())
        q, scale = _exact_codes(y, torch.float8_e4m3fn, 1)
        return {"h": h, "y": y if case["y"] else None, "rstd": rstd, "q": q, "scales": scale}
    if case["op"] == "norm_backward":
        h, dy, w, r = s["h"].double(), s["dy"].double(), s["weight"].double(), s["rstd"].double()
        dot = torch.mv(h * dy, w)  # sum of dy w h of each row
        dx = r[:, None] * dy * w - (r.pow(3) * dot / h.shape[1])[:, None] * h
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return {"dx": dx, "dweight": torch.mv((dy * h).t(), r)}
    b_rows = case["block_rows"]
    a = s["a"].double() * s["a_scales"].double().repeat_interleave(GROUP, 1)[:, :case["k"]]
    wide = s["b_scales"].double().repeat_interleave(b_rows, 0)[:case["n"]]
    b = s["b"].double() * wide.repeat_interleave(GROUP, 1)[:, :case["k"]]
    return {"out": a @ b.t()}
