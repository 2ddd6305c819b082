"""Cases of the operators that a training step runs around its layers' products: the
global gradient norm over many tensors (zr_grad_norm), clipping by it in place
(zr_clip_grads) and inside AdamW (zr_adamw_step_clip), and the norm of queries and keys
for each head with the rotation by their positions (zr_qk_norm_rope) with its backward
pass (zr_qk_norm_rope_backward).

A clip record is 16 bytes of device memory: the sum of squares (fp64), the norm and the
factor (fp32).  Queries and keys are slices of the rows that a fused query/key/value
product leaves: [tokens, (q heads + 2 * k heads) * head_dim].
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HPARAMS = dict(lr=5e-5, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
GRAD_STD = 1e-3
NORM_EPS = 1e-5   # of the head norms
CLIP_EPS = 1e-6   # beside the gradient norm
PARTIALS = 2048   # sums in the gradient norm's workspace
GRAD_PARTIALS = 512  # rows of partial sums in the rotation's backward workspace


def listed():
    return [
        # The 65 norm vectors of a 7B model, which stay whole on every rank: latency.
        {"name": "norm_vectors", "op": "norm", "tensors": "norms", "count": 65, "type": "bf16"},
        # Unreduced fp32 gradients of four decoder layers, norms and matrices mixed.
        {"name": "norm_layers", "op": "norm", "tensors": "layers", "count": 4, "type": "fp32"},
        # The reduced gradient shard of a 7B model over 4 ranks, one flat buffer.
        {"name": "norm_shard", "op": "norm", "tensors": "flat", "count": 1_750_000_000, "type": "bf16"},
        # Biases and norm vectors of a GPT-style model of 36 layers.
        {"name": "clip_vectors", "op": "clip", "tensors": "vectors", "count": 36, "type": "bf16"},
        # Gradients of two decoder layers in fp16.
        {"name": "clip_layers", "op": "clip", "tensors": "layers", "count": 2, "type": "fp16"},
        # The shard of a small model: latency.
        {"name": "adamw_small", "op": "adamw", "count": 262_144, "type": "bf16"},
        # A 7B model's shard over 64 ranks.
        {"name": "adamw_shard", "op": "adamw", "count": 105_283_584, "type": "bf16"},
        # One decoded token, 128K into its context: latency.
        {"name": "rope_token", "op": "rope", "tokens": 1, "q_heads": 32, "k_heads": 8, "head_dim": 128, "rot_dim": 128,
         "axes": 1, "interleaved": False, "type": "bf16", "far": 131_000},
        # A training batch of packed documents.
        {"name": "rope_training", "op": "rope", "tokens": 16384, "q_heads": 32, "k_heads": 8, "head_dim": 128,
         "rot_dim": 128, "axes": 1, "interleaved": False, "type": "bf16", "far": 0},
        # A ragged batch of video patches: time, height and width.
        {"name": "rope_video", "op": "rope", "tokens": 5003, "q_heads": 20, "k_heads": 4, "head_dim": 96, "rot_dim": 96,
         "axes": 3, "interleaved": True, "type": "fp16", "far": 0},
        # Backward of a small ragged batch, a quarter of each head rotated.
        {"name": "rope_backward_small", "op": "rope_backward", "tokens": 777, "q_heads": 16, "k_heads": 4, "head_dim": 80,
         "rot_dim": 20, "axes": 1, "interleaved": False, "type": "fp16", "far": 0},
        # Backward of the training batch.
        {"name": "rope_backward", "op": "rope_backward", "tokens": 16384, "q_heads": 32, "k_heads": 8, "head_dim": 128,
         "rot_dim": 128, "axes": 1, "interleaved": False, "type": "bf16", "far": 0},
    ]


def _spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "clip", "adamw", "rope", "rope", "rope_backward", "rope_backward"])
    if op in ("norm", "clip"):
        kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        tensors = rng.choice(["norms", "vectors", "layers", "flat", "ragged"])
        count = {"norms": lambda: rng.randint(1, 129), "vectors": lambda: rng.randint(1, 96),
                 "layers": lambda: rng.randint(1, 2), "flat": lambda: _spread(rng, 1, 400_000_000),
                 "ragged": lambda: rng.randint(1, 600)}[tensors]()
        return {"op": op, "tensors": tensors, "count": count, "type": kind}
    if op == "adamw":
        return {"op": op, "count": _spread(rng, 1, 105_283_584), "type": rng.choice(["bf16", "bf16", "fp16"])}
    dim = rng.choice([64, 64, 72, 80, 96, 128, 128, 128, 256])
    rot = rng.choice([dim, dim, dim // 2, dim // 4 // 2 * 2])
    q = rng.choice([8, 12, 16, 20, 28, 32, 40, 64])
    k = q // rng.choice([1, 2, 4, 4])
    return {"op": op, "tokens": _spread(rng, 1, 83_000_000 // ((q + k) * dim)), "q_heads": q, "k_heads": k, "head_dim": dim,
            "rot_dim": rot, "axes": rng.choice([1, 1, 2, 3]), "interleaved": rng.random() < 0.3,
            "type": rng.choice(["bf16", "bf16", "fp16"]), "far": rng.choice([0, 0, 131_000, 1_000_000])}


def _sizes(case):
    """Elements of each tensor of a list, in the order of the model's layers."""
    kind, n = case["tensors"], case["count"]
    hidden, ffn = 4096, 11008
    if kind == "flat":
        return [n]
    if kind == "norms":
        return [hidden] * n
    if kind == "vectors":
        return [hidden, hidden, 3 * hidden, hidden, hidden, hidden, 4 * hidden, hidden] * n + [hidden, hidden]
    if kind == "layers":
        return ([hidden * hidden] * 4 + [hidden * ffn] * 3 + [hidden] * 2) * n
    # lengths of every kind, one and odd ones among them, so that tensors start at any element of the flat buffer
    return [1 + (i * 7919 + n) % 5003 + (200_003 if i % 29 == 7 else 0) for i in range(n)]


def _axis_of(case):
    """The axis whose position turns each pair: as even a split as there is, one axis after the other."""
    half = case["rot_dim"] // 2
    return [j * case["axes"] // half for j in range(half)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    op, kind = case["op"], TYPES[case["type"]]
    s = dict(case)
    if op in ("norm", "clip", "adamw"):
        # sum of squares, norm and factor of an earlier norm: 2.7 clipped to 1
        s["clip"] = torch.tensor([7.29, 0.0], dtype=torch.float64, device="cuda")
        s["clip"].view(torch.float32)[2:] = torch.tensor([2.7, 1 / 2.7], device="cuda")
    if op in ("norm", "clip"):
        sizes = _sizes(case)
        # fp16 gradients carry a loss scale
        s["flat"] = randn(sum(sizes)).mul_(GRAD_STD * (1024 if kind == torch.float16 else 1)).to(kind)
        s["grads"] = list(torch.split(s["flat"], sizes))
        s["workspace"] = torch.empty(PARTIALS, dtype=torch.float64, device="cuda")
        s["max_norm"] = 1.0
        if own:
            import zero_sharded_optimizer_zr_amd as zr
            s["list"] = zr.tensor_list(s["grads"])  # kept by a program from step to step
        return s
    if op == "adamw":
        n = case["count"]
        s["master"], s["m"] = randn(n) * 0.02, randn(n) * 1e-4
        s["v"] = torch.rand(n, generator=g, device="cuda") * 1e-6
        s["scale"] = 1024.0 if kind == torch.float16 else 1.0
        s["grad"] = (randn(n) * GRAD_STD * s["scale"]).to(kind)
        s["param"] = torch.empty(n, dtype=kind, device="cuda")
        # scale, clean steps, overflow flag, skipped steps
        s["ls"] = torch.zeros(4, dtype=torch.int32, device="cuda")
        s["ls"].view(torch.float32)[0] = s["scale"]
        return s
    t, hq, hk, d, rot = (case[x] for x in ("tokens", "q_heads", "k_heads", "head_dim", "rot_dim"))
    # tokens' sizes differ from one to the next
    rows = (randn(t, (hq + 2 * hk) * d) * torch.exp(0.5 * randn(t, 1))).to(kind)
    split = lambda x: (x[:, :hq * d].view(t, hq, d), x[:, hq * d:(hq + hk) * d].view(t, hk, d))  # noqa: E731
    s["q"], s["k"] = split(rows)
    s["q_weight"], s["k_weight"] = ((1 + 0.1 * randn(d)).to(kind) for _ in "qk")
    index = torch.arange(t, device="cuda")
    # documents of 4096 tokens, or one context that begins far on; frames of 24 x 36 patches
    text = (index + case["far"]) if case["far"] else index % 4096
    grid = [text // 864, text % 864 // 36, text % 36]
    s["positions"] = torch.stack(grid[:case["axes"]]).contiguous() if case["axes"] > 1 else text
    base = 1e6 if case["far"] else 1e4
    s["inv_freq"] = (base ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(1, rot))).float()
    new = lambda h: torch.empty(t, h, d, dtype=kind, device="cuda")  # noqa: E731
    if op == "rope":
        s["q_out"], s["k_out"] = new(hq), new(hk)
    else:
        s["dq"], s["dk"] = (randn(t, h, d).to(kind) for h in (hq, hk))
        # gradients of the fused product's rows
        s["dq_in"], s["dk_in"] = split(torch.empty(t, (hq + 2 * hk) * d, dtype=kind, device="cuda"))
        s["dq_weight"], s["dk_weight"] = (torch.empty(d, dtype=kind, device="cuda") for _ in "qk")
        s["workspace"] = torch.empty(GRAD_PARTIALS, d, dtype=torch.float32, device="cuda")
    if own:
        import zero_sharded_optimizer_zr_amd as zr
        s["rope"] = zr.rope(s["inv_freq"], interleaved=case["interleaved"], pair_axis=_axis_of(case))
    return s


def _record(clip):
    return {"sum_squares": clip[0], "norm": clip.view(torch.float32)[2], "factor": clip.view(torch.float32)[3]}


def _run_own(s):
    import zero_sharded_optimizer_zr_amd as zr
    if s["op"] == "norm":
        zr.zr_grad_norm(s["list"], s["clip"], s["workspace"], max_norm=s["max_norm"], eps=CLIP_EPS)
        return _record(s["clip"])
    if s["op"] == "clip":
        zr.zr_clip_grads(s["list"], s["clip"])
        return {"grads": s["flat"]}
    if s["op"] == "adamw":
        state = (s["grad"], s["master"], s["m"], s["v"], s["param"])
        if s["type"] == "fp16":
            zr.zr_adamw_step_clip_f16(*state, s["ls"], s["clip"], step=10, **HPARAMS)
        else:
            zr.zr_adamw_step_clip(*state, s["clip"], step=10, **HPARAMS)
        return {"master": s["master"], "exp_avg": s["m"], "exp_avg_sq": s["v"], "param": s["param"]}
    place = (s["q_weight"], s["k_weight"], s["positions"], s["rope"])
    if s["op"] == "rope":
        zr.zr_qk_norm_rope(s["q"], s["k"], *place, s["q_out"], s["k_out"], eps=NORM_EPS)
        return {"q": s["q_out"], "k": s["k_out"]}
    zr.zr_qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], *place, s["dq_in"], s["dk_in"], s["dq_weight"],
                                s["dk_weight"], s["workspace"], eps=NORM_EPS)
    return {"dq": s["dq_in"], "dk": s["dk_in"], "dq_weight": s["dq_weight"], "dk_weight": s["dk_weight"]}


def _turns(s):
    """Cosine and sine of every token's pairs; the angles of far positions lose too much in 32 bits."""
    positions = s["positions"].view(-1, s["tokens"])
    if s["rot_dim"] == 0:
        return torch.ones(s["tokens"], 1, 0, device="cuda"), torch.zeros(s["tokens"], 1, 0, device="cuda")
    at = positions[torch.tensor(_axis_of(s), device="cuda")]
    angle = at.t().double() * s["inv_freq"].double()
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _pairs(x, rot, interleaved):
    """First and second elements of the pairs of x's last axis, and the rest, which is not turned."""
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _joined(a, b, rest, interleaved):
    turned = torch.stack((a, b), dim=-1).flatten(-2) if interleaved else torch.cat((a, b), dim=-1)
    return torch.cat((turned, rest), dim=-1)


def _run_plain(s):
    if s["op"] == "norm":  # a sum over up to 2^31 elements: in 64 bits
        total = torch.stack([g.double().square().sum() for g in s["grads"]]).sum()
        norm = torch.sqrt(total)
        factor = torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0)
        return {"sum_squares": total, "norm": norm.float(), "factor": factor.float()}
    if s["op"] == "clip":
        factor = s["clip"].view(torch.float32)[3]
        for g in s["grads"]:
            g.copy_(g.float() * factor)
        return {"grads": s["flat"]}
    if s["op"] == "adamw":
        # In 64 bits, each state rounded once: where the decayed parameter and the step nearly cancel, 32 lose the
        # 16-bit copy's last places.
        lr, b1, b2, eps, wd = (HPARAMS[k] for k in ("lr", "beta1", "beta2", "eps", "weight_decay"))
        g = s["grad"].double() * (1 / s["scale"]) * s["clip"].view(torch.float32)[3].double()
        m = b1 * s["m"].double() + (1 - b1) * g
        v = b2 * s["v"].double() + (1 - b2) * g * g
        step = lr * (m / (1 - b1 ** 10)) / (torch.sqrt(v / (1 - b2 ** 10)) + eps)
        s["master"].copy_(s["master"].double() * (1 - lr * wd) - step)
        s["m"].copy_(m)
        s["v"].copy_(v)
        s["param"].copy_(s["master"])
        return {"master": s["master"], "exp_avg": s["m"], "exp_avg_sq": s["v"], "param": s["param"]}
    cos, sin = _turns(s)
    rot, inter = s["rot_dim"], s["interleaved"]
    out = {}
    for name in "qk":
        x, w, kind = s[name].float(), s[name + "_weight"].float(), s[name].dtype
        rstd = torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + NORM_EPS)
        if s["op"] == "rope":
            a, b, rest = _pairs(x * rstd * w, rot, inter)
            out[name] = _joined(a * cos - b * sin, b * cos + a * sin, rest, inter).to(kind)
            continue
        a, b, rest = _pairs(s["d" + name].float(), rot, inter)
        g = _joined(a * cos + b * sin, b * cos - a * sin, rest, inter)
        xh = x * rstd
        out[f"d{name}_weight"] = (g * xh).sum(dim=(0, 1)).to(kind)
        g = g * w
        out["d" + name] = (rstd * (g - xh * (g * xh).mean(dim=-1, keepdim=True))).to(kind)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, size = case["op"], 4 if case["type"] == "fp32" else 2
    if op in ("norm", "clip"):
        n = sum(_sizes(case))
        return {"bytes": n * size * (2 if op == "clip" else 1) + 16, "flops": n * (1 if op == "clip" else 2)}
    if op == "adamw":
        return {"bytes": 28 * case["count"] + 16, "flops": 15 * case["count"]}
    n = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["head_dim"]
    other = case["tokens"] * case["axes"] * 8 + case["rot_dim"] * 2 + 2 * size * case["head_dim"]
    if op == "rope":
        return {"bytes": 2 * n * size + other, "flops": 8 * n}
    return {"bytes": 3 * n * size + other + 2 * size * case["head_dim"], "flops": 16 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        total = sum(float(torch.dot(part, part)) for g in s["grads"] for part in
                    (p.double() for p in torch.split(g, 1 << 27)))
        norm = math.sqrt(total)
        value = lambda x: torch.tensor(x, dtype=torch.float64)  # noqa: E731
        return {"sum_squares": value(total), "norm": value(norm), "factor": value(min(1.0, s["max_norm"] / (norm + CLIP_EPS)))}
    factor = s["clip"].view(torch.float32)[3].item() if "clip" in s else None
    if case["op"] == "clip":
        return {"grads": s["flat"].double() * factor}
    if case["op"] == "adamw":
        hp, t = HPARAMS, 10
        g = s["grad"].double() / s["scale"] * factor
        m = torch.lerp(g, s["m"].double(), hp["beta1"])
        v = torch.lerp(g.square(), s["v"].double(), hp["beta2"])
        bias = math.sqrt(1 - hp["beta2"] ** t)
        move = hp["lr"] * bias / (1 - hp["beta1"] ** t) * m / (v.sqrt() + hp["eps"] * bias)
        master = s["master"].double() * (1 - hp["lr"] * hp["weight_decay"]) - move
        return {"master": master, "exp_avg": m, "exp_avg_sq": v, "param": master}
    # pairs as complex numbers, turned by a product with exp(i angle)
    rot, inter, half = case["rot_dim"], case["interleaved"], case["rot_dim"] // 2
    positions = s["positions"].view(-1, case["tokens"]).double()
    angle = torch.empty(case["tokens"], half, dtype=torch.float64, device="cuda")
    for j, axis in enumerate(_axis_of(case)):
        angle[:, j] = positions[axis] * s["inv_freq"][j].double()
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]

    def turned(x, by):
        x = x.clone()
        z = x[..., :rot].unflatten(-1, (half, 2)) if inter else x[..., :rot].unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * by)
        x[..., :rot] = (z if inter else z.transpose(-1, -2)).flatten(-2)
        return x

    out = {}
    for name in "qk":
        x, w = s[name].double(), s[name + "_weight"].double()
        size = torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + NORM_EPS)
        if case["op"] == "rope":
            out[name] = turned(x / size * w, turn) if rot else x / size * w
            continue
        g = turned(s["d" + name].double(), turn.conj()) if rot else s["d" + name].double()
        out[f"d{name}_weight"] = (g * x / size).flatten(0, 1).sum(0)
        along = (g * w * x).sum(-1, keepdim=True) / x.shape[-1]
        out["d" + name] = g * w / size - x * along / size.pow(3)
    return out
