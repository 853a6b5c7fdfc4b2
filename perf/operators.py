"""Cases of the dense operators: products with packed 4-bit weights and the gated feed-forward block.

Four operators, each in its plain form (elementary torch operations in 32 bits)
and, with `own` set, through the framework's calls:

  linear    y = W x (+ b), W packed: 4-bit codes under block scales
  gated     h = silu(W_gate x) * (W_up x), gate and up rows of W interleaved, packed
  ffn       y = W_down (silu(W_gate x) * (W_up x)), 16-bit weights
  ffn_grad  gradients of `ffn` by x, W_gate/W_up (interleaved) and W_down

Packed formats: one fp16 scale per 32 or per 128 elements of a row, or one E4M3
byte per 32 elements under one fp32 scale per row; a code c stands for c - 8, or
for c - 7.5 with half-integer levels.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one eight-token step through the smallest projection of the tests' layer: launch latency
        {"name": "linear_t8_256x256", "op": "linear", "tokens": 8, "rows": 256, "cols": 256, "block": 32, "half": False,
         "fp8": False, "x": "bf16", "y": "bf16", "bias": False},
        # an attention-sized projection at the framework's hidden size, one token
        {"name": "linear_t1_2048x2048", "op": "linear", "tokens": 1, "rows": 2048, "cols": 2048, "block": 32,
         "half": False, "fp8": False, "x": "bf16", "y": "bf16", "bias": True},
        # a vocabulary head, odd row count, fp32 logits for four sequences
        {"name": "linear_t4_100003x2048", "op": "linear", "tokens": 4, "rows": 100003, "cols": 2048, "block": 32,
         "half": False, "fp8": False, "x": "bf16", "y": "fp32", "bias": False},
        # a batch of 16 through a wide down projection, groups of 128, fp16 activations
        {"name": "linear_t16_4097x8192_g128", "op": "linear", "tokens": 16, "rows": 4097, "cols": 8192, "block": 128,
         "half": False, "fp8": False, "x": "fp16", "y": "fp16", "bias": True},
        # the largest decode batch, fp8 block scales, columns that are no multiple of 256
        {"name": "linear_t64_8192x4128_fp8", "op": "linear", "tokens": 64, "rows": 8192, "cols": 4128, "block": 32,
         "half": False, "fp8": True, "x": "bf16", "y": "bf16", "bias": False},
        # the shared expert's gate and up projections for one token
        {"name": "gated_t1_768x2048", "op": "gated", "tokens": 1, "rows": 768, "cols": 2048, "block": 32, "half": False,
         "fp8": False, "x": "bf16", "y": "bf16"},
        # a dense block's gate and up projections for a batch of 16, half-integer levels
        {"name": "gated_t16_10240x4096_half", "op": "gated", "tokens": 16, "rows": 10240, "cols": 4096, "block": 32,
         "half": True, "fp8": False, "x": "bf16", "y": "bf16"},
        # one token through the 16-bit block at the shared expert's size
        {"name": "ffn_t1_2048x768", "op": "ffn", "tokens": 1, "hidden": 2048, "inter": 768, "x": "bf16"},
        # a ragged fp16 batch, sizes that fill no tile
        {"name": "ffn_t777_2056x5000_fp16", "op": "ffn", "tokens": 777, "hidden": 2056, "inter": 5000, "x": "fp16"},
        # a training batch through a dense block
        {"name": "ffn_t8192_2048x8192", "op": "ffn", "tokens": 8192, "hidden": 2048, "inter": 8192, "x": "bf16"},
        # gradients of an odd small batch at the shared expert's size
        {"name": "grad_t257_2048x768", "op": "ffn_grad", "tokens": 257, "hidden": 2048, "inter": 768, "x": "bf16"},
        # gradients of the training batch
        {"name": "grad_t8192_2048x8192", "op": "ffn_grad", "tokens": 8192, "hidden": 2048, "inter": 8192, "x": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "gated", "ffn", "ffn_grad"])
    x = rng.choice(["bf16", "fp16"])
    if op in ("linear", "gated"):
        fmt = rng.choice(["32", "32", "128", "half", "half128", "fp8"])
        block = 128 if fmt.endswith("128") else 32
        tokens = _log(rng, 1, 64)
        cols = block * _log(rng, 256 // block, 8192 // block)
        most = min(100003 if op == "linear" else 20000, 1600000000 // (tokens * cols), 200000000 // cols)
        rows = _log(rng, 17, max(64, most))
        c = {"op": op, "tokens": tokens, "rows": rows, "cols": cols, "block": block, "half": fmt.startswith("half"),
             "fp8": fmt == "fp8", "x": x, "y": rng.choice([x, "fp32"])}
        if op == "linear":
            c["bias"] = rng.random() < 0.5
        return c
    tokens = _log(rng, 1, 8192)
    hidden = 8 * _log(rng, 16, 512)
    inter = 8 * _log(rng, 16, min(1376, max(16, 8192 * 2048 * 8192 // (8 * tokens * hidden))))
    return {"op": op, "tokens": tokens, "hidden": hidden, "inter": inter, "x": x}


def _packed(case, gen, rows):
    """Codes and scales of a [rows, cols] matrix of N(0, 0.02) weights, quantised symmetrically per block."""
    block = case["block"]
    levels = 7.5 if case["half"] else 7.0
    w = torch.randn(rows, case["cols"] // block, block, generator=gen, device="cuda") * 0.02
    top = w.abs().amax(2)
    if case["fp8"]:
        row_scales = top.amax(1) / (levels * 448.0)
        scales = (top / (levels * row_scales[:, None])).to(torch.float8_e4m3fn)
        s = scales.float() * row_scales[:, None]
        scales = scales.view(torch.uint8)
    else:
        row_scales = None
        scales = (top / levels).half()
        s = scales.float()
    w /= s[:, :, None]
    c = torch.floor(w) + 8 if case["half"] else torch.round(w).clamp(-7, 7) + 8
    c = c.clamp(0, 15).to(torch.uint8).view(rows, -1, 2)
    codes = c[:, :, 0] | (c[:, :, 1] << 4)
    return codes, scales, row_scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    xt = TYPES[case["x"]]
    s = {"case": case}
    t = case["tokens"]
    if case["op"] in ("linear", "gated"):
        rows = case["rows"] * (2 if case["op"] == "gated" else 1)
        s["codes"], s["scales"], s["row_scales"] = _packed(case, gen, rows)
        s["x"] = torch.randn(t, case["cols"], generator=gen, device="cuda").to(xt)
        s["y"] = torch.empty(t, case["rows"], dtype=TYPES[case["y"]], device="cuda")
        if case.get("bias"):
            s["bias"] = torch.randn(rows, generator=gen, device="cuda") * 0.1
        return s
    h, i = case["hidden"], case["inter"]
    s["x"] = torch.randn(t, h, generator=gen, device="cuda").to(xt)
    s["w_gate_up"] = (torch.randn(2 * i, h, generator=gen, device="cuda") * 0.02).to(xt)
    s["w_down"] = (torch.randn(h, i, generator=gen, device="cuda") * 0.02).to(xt)
    if case["op"] == "ffn":
        s["y"] = torch.empty(t, h, dtype=xt, device="cuda")
    else:
        s["dy"] = (torch.randn(t, h, generator=gen, device="cuda") * 0.0625).to(xt)
        s["dx"] = torch.empty(t, h, dtype=xt, device="cuda")
        s["dw_gate_up"] = torch.empty(2 * i, h, dtype=xt, device="cuda")
        s["dw_down"] = torch.empty(h, i, dtype=xt, device="cuda")
    return s


def _weights(s, dtype):
    """The packed matrix as numbers of `dtype`, [rows, cols]."""
    case, codes = s["case"], s["codes"]
    q = torch.stack((codes & 15, codes >> 4), 2).view(codes.shape[0], -1, case["block"]).to(dtype)
    q = q - (7.5 if case["half"] else 8.0)
    if case["fp8"]:
        b = s["scales"].view(torch.float8_e4m3fn).to(dtype) * s["row_scales"].to(dtype)[:, None]
    else:
        b = s["scales"].to(dtype)
    return (q * b[:, :, None]).view(codes.shape[0], -1)


def _run_own(s):
    import quantized_expert_ffn_moe_b200 as q
    case = s["case"]
    if case["op"] in ("linear", "gated"):
        if "cfg" not in s:
            s["cfg"] = q.linear_config_of(4, case["block"], half_levels=case["half"], fp8_scales=case["fp8"])
        if case["op"] == "linear":
            q.moe_linear_forward(s["cfg"], s["codes"], s["scales"], s["x"], s["y"], row_scales=s["row_scales"],
                                 bias=s.get("bias"))
        else:
            q.moe_linear_gated_forward(s["cfg"], s["codes"], s["scales"], s["x"], s["y"], row_scales=s["row_scales"])
        return s["y"]
    t, h, i = case["tokens"], case["hidden"], case["inter"]
    if "workspace" not in s:
        n = q.moe_ffn_workspace_bytes(h, i, t, backward=case["op"] == "ffn_grad")
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    if case["op"] == "ffn":
        q.moe_ffn_forward(s["w_gate_up"], s["w_down"], s["x"], s["y"], s["workspace"])
        return s["y"]
    q.moe_ffn_backward(s["w_gate_up"], s["w_down"], s["x"], s["dy"], s["workspace"], dx=s["dx"],
                       dw_gate_up=s["dw_gate_up"], dw_down=s["dw_down"])
    return {"dx": s["dx"], "dw_gate_up": s["dw_gate_up"], "dw_down": s["dw_down"]}


def run(state):
    s = state
    if own:
        return _run_own(s)
    case = s["case"]
    xt = TYPES[case["x"]]
    x = s["x"].float()
    if case["op"] == "linear":
        y = x @ _weights(s, torch.float32).T
        if "bias" in s:
            y = y + s["bias"]
        return y.to(TYPES[case["y"]])
    if case["op"] == "gated":
        z = x @ _weights(s, torch.float32).T
        g, u = z[:, 0::2], z[:, 1::2]
        return (g / (1 + torch.exp(-g)) * u).to(TYPES[case["y"]])
    wgu, wd = s["w_gate_up"].float(), s["w_down"].float()
    z = x @ wgu.T
    g, u = z[:, 0::2], z[:, 1::2]
    sig = 1 / (1 + torch.exp(-g))
    a = g * sig
    hid = a * u
    if case["op"] == "ffn":
        return (hid @ wd.T).to(xt)
    dy = s["dy"].float()
    dh = dy @ wd
    dz = torch.empty_like(z)
    dz[:, 0::2] = dh * u * (sig + a * (1 - sig))
    dz[:, 1::2] = dh * a
    return {"dx": (dz @ wgu).to(xt), "dw_gate_up": (dz.T @ x).to(xt), "dw_down": (dy.T @ hid).to(xt)}


def work(case):
    t = case["tokens"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if case["op"] in ("linear", "gated"):
        n = case["rows"] * (2 if case["op"] == "gated" else 1)
        k = case["cols"]
        b = n * k // 2 + n * (k // case["block"]) * (1 if case["fp8"] else 2) + (4 * n if case["fp8"] else 0)
        b += t * k * 2 + t * case["rows"] * size[case["y"]] + (4 * n if case.get("bias") else 0)
        return {"bytes": b, "flops": 2 * t * n * k}
    h, i = case["hidden"], case["inter"]
    if case["op"] == "ffn":
        return {"bytes": 2 * (3 * h * i + 2 * t * h), "flops": 6 * t * h * i}
    return {"bytes": 2 * (6 * h * i + 3 * t * h), "flops": 16 * t * h * i}


def exact(case, seed):
    """The same from the definition in 64 bits: sums over blocks for the packed products, autograd for the gradients."""
    s = prepare(case, seed)
    x = s["x"].double()
    t = case["tokens"]
    if case["op"] in ("linear", "gated"):
        n, k, block = s["codes"].shape[0], case["cols"], case["block"]
        z = torch.empty(t, n, dtype=torch.float64, device=x.device)
        xb = x.view(t, k // block, block)
        for r0 in range(0, n, 2048):
            c = s["codes"][r0:r0 + 2048].long()
            q = torch.empty(c.shape[0], k, dtype=torch.float64, device=x.device)
            q[:, 0::2] = (c % 16).double()
            q[:, 1::2] = (c // 16).double()
            q -= 7.5 if case["half"] else 8.0
            if case["fp8"]:
                b = s["scales"][r0:r0 + 2048].long()
                e, m = (b >> 3) & 15, (b & 7).double()
                v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
                v = torch.where(b >= 128, -v, v) * s["row_scales"][r0:r0 + 2048].double()[:, None]
            else:
                v = s["scales"][r0:r0 + 2048].double()
            q = q.view(-1, k // block, block)
            part = torch.einsum("tbk,nbk->tnb", xb, q) if t * c.shape[0] * (k // block) < 1 << 28 else None
            if part is None:
                z[:, r0:r0 + 2048] = x @ (q * v[:, :, None]).view(-1, k).T
            else:
                z[:, r0:r0 + 2048] = (part * v[None]).sum(2)
        if case["op"] == "linear":
            return z + s["bias"].double() if "bias" in s else z
        g = z[:, 0::2]
        return torch.nn.functional.silu(g) * z[:, 1::2]
    grad = case["op"] == "ffn_grad"
    wgu, wd = s["w_gate_up"].double(), s["w_down"].double()
    leaves = [v.requires_grad_(grad) for v in (x, wgu, wd)]
    y = (torch.nn.functional.silu(x @ wgu[0::2].T) * (x @ wgu[1::2].T)) @ wd.T
    if not grad:
        return y
    dx, dw_gate_up, dw_down = torch.autograd.grad(y, leaves, s["dy"].double())
    return {"dx": dx, "dw_gate_up": dw_gate_up, "dw_down": dw_down}
