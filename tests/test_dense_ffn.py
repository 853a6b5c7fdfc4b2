"""The dense gated feed-forward block on 16-bit weights (moe_ffn_forward) and
its gradients (moe_ffn_backward) against the definition in 64 bits."""
import numpy as np
import pytest

import quantized_expert_ffn_moe_b200 as q
from quantized_expert_ffn_moe_b200 import build as qbuild


# ------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return q.load_library()


A = 1 << 30          # never dereferenced: every call below is refused or launches nothing


def fwd(lib, H=64, I=64, ty=q.MOE_BF16, wgu=A, wd=2 * A, x=3 * A, T=4, y=4 * A, ws=5 * A, n=1 << 40):
    return lib.moe_ffn_forward(H, I, ty, wgu, wd, x, T, y, ws, n, None)


def bwd(lib, H=64, I=64, ty=q.MOE_BF16, wgu=A, wd=2 * A, x=3 * A, dy=4 * A, T=4, dx=6 * A, dwgu=7 * A, dwd=8 * A,
        ws=5 * A, n=1 << 29):
    return lib.moe_ffn_backward(H, I, ty, wgu, wd, x, dy, T, dx, dwgu, dwd, ws, n, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_refusals(lib, call):
    kw = dict(n=1 << 29)
    for bad in (dict(H=0), dict(I=0), dict(H=-8), dict(T=-1), dict(ty=q.MOE_FP32), dict(ty=5), dict(wgu=None),
                dict(wd=None), dict(x=None), dict(x=3 * A + 8), dict(wgu=A + 2), dict(ws=None), dict(ws=5 * A + 16)):
        assert call(lib, **{**kw, **bad}) == -1, bad
    for bad in (dict(H=60), dict(I=4), dict(H=65544), dict(I=65544), dict(T=(1 << 22) + 1)):
        assert call(lib, **{**kw, **bad}) == -2, bad
    need = q.moe_ffn_workspace_bytes(64, 64, 4, backward=call is bwd)
    assert need > 0 and call(lib, n=need - 1) == -3
    outs = ["y"] if call is fwd else ["dx", "dwgu", "dwd"]
    for o in outs:
        assert call(lib, **kw, **{o: 9 * A + 4}) == -1
        for taken in (A, 2 * A, 3 * A, 5 * A):
            assert call(lib, **kw, **{o: taken + 16}) == -1, (o, taken)
    assert call(lib, **kw, ws=3 * A) == -1                                    # workspace over x
    if call is fwd:
        assert fwd(lib, y=None) == -1
        assert fwd(lib, T=0, x=None, y=None, ws=None, wgu=None) == 0
    else:
        assert bwd(lib, dy=None) == -1
        assert bwd(lib, dx=7 * A) == -1                                       # two outputs in one place
        assert bwd(lib, dx=None, dwgu=None, dwd=None) == 0                    # nothing asked for
        assert bwd(lib, T=0, dx=None, dwgu=None, dwd=None, ws=None) == 0


def test_workspace_bytes(lib):
    f, b = (q.moe_ffn_workspace_bytes(2048, 768, 100, backward=v) for v in (False, True))
    assert f >= 100 * 768 * 2 and b >= 3 * 100 * 768 * 2 and b > f
    for bad in ((0, 8, 1), (8, 0, 1), (8, 12, 1), (8, 8, -1), (65544, 8, 1)):
        assert q.moe_ffn_workspace_bytes(*bad) == 0


def test_binding_refusals(lib):
    torch = pytest.importorskip("torch")
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)  # noqa: E731
    good = dict(w_gate_up=z(32, 64), w_down=z(64, 16), x=z(3, 64), y=z(3, 64))
    for bad in (dict(w_gate_up=z(16, 64)), dict(y=z(2, 64)), dict(y=z(3, 64, d=torch.float16)), dict(x=z(64, 3).T),
                dict(w_down=z(64, 16, d=torch.float16)), dict(x=z(3, 64, d=torch.float32)), {}):
        a = {**good, **bad}
        with pytest.raises(ValueError):          # the last one: tensors of the host
            q.moe_ffn_forward(a["w_gate_up"], a["w_down"], a["x"], a["y"], z(1))
    with pytest.raises(ValueError):
        q.moe_ffn_backward(good["w_gate_up"], good["w_down"], good["x"], z(2, 64), z(1))
    with pytest.raises(ValueError):
        q.moe_ffn_backward(good["w_gate_up"], good["w_down"], good["x"], z(3, 64), z(1), dw_down=z(16, 64))


# -------------------------------------------------- the formula itself
def ref_forward(x, wgu, wd):
    g, u = x @ wgu[0::2].T, x @ wgu[1::2].T
    return (g / (1 + np.exp(-g)) * u) @ wd.T


def ref_backward(x, wgu, wd, dy):
    g, u = x @ wgu[0::2].T, x @ wgu[1::2].T
    s = 1 / (1 + np.exp(-g))
    a = g * s
    dh = dy @ wd
    dgu = np.empty((x.shape[0], wgu.shape[0]))
    dgu[:, 0::2], dgu[:, 1::2] = dh * u * (s + a * (1 - s)), dh * a
    return dgu @ wgu, dgu.T @ x, dy.T @ (a * u)


def test_formula_against_differences():
    r = np.random.default_rng(0)
    v = [r.normal(size=s) * c for s, c in (((5, 16), 1.0), ((24, 16), 0.4), ((16, 12), 0.4))]
    dy = r.normal(size=(5, 16))
    grads = ref_backward(*v, dy)
    for k in range(3):
        d = r.normal(size=v[k].shape)
        e = 1e-5
        plus, minus = (ref_forward(*[w + (sg * e * d if i == k else 0) for i, w in enumerate(v)]) for sg in (1, -1))
        want = ((plus - minus) * dy).sum() / (2 * e)
        assert abs((grads[k] * d).sum() - want) <= 1e-7 * np.abs(grads[k] * d).sum()


# ------------------------------------------------------------ on the GPU
gpu = pytest.mark.gpu

SHAPES = [
    # T, H, I: single tokens, sizes around the tiles' edges (128 x 64 and 256 x 256), sizes of one 16-byte unit
    (1, 8, 8), (1, 2048, 768), (2, 64, 64), (7, 72, 40), (63, 128, 120), (64, 64, 136), (65, 256, 128), (127, 200, 64),
    (128, 128, 64), (129, 136, 72), (257, 512, 1000), (300, 2048, 768),
    # wide tiles: full, and ragged in every direction
    (512, 2048, 4096), (1111, 1000, 3144), (2049, 2056, 1032),
    # a tile's reduction split over a cluster: by 4 and 2 on narrow tiles, over two pairs on wide ones, uneven parts
    (5, 1032, 520), (100, 2048, 256), (130, 776, 1096), (777, 2056, 5000), (500, 1024, 4104),
    # few tokens (the rest of h's and dgu's rounding is kept) on either tile
    (64, 1024, 4096), (33, 4096, 8000), (16, 2048, 8192),
]


def inputs(T, H, I, dtype, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda *s, c=1.0: (torch.randn(*s, generator=g, device="cuda") * c).to(dtype)  # noqa: E731
    return mk(T, H), mk(2 * I, H, c=0.7 / H ** 0.5), mk(H, I, c=0.7 / I ** 0.5), mk(T, H, c=0.1)


def torch_ref(x, wgu, wd, dy=None):
    import torch
    x, wgu, wd = x.double(), wgu.double(), wd.double()
    g, u = x @ wgu[0::2].T, x @ wgu[1::2].T
    s = torch.sigmoid(g)
    a = g * s
    h = a * u
    if dy is None:
        return h @ wd.T, h.abs() @ wd.abs().T
    dy = dy.double()
    dh = dy @ wd
    dgu = torch.empty(x.shape[0], wgu.shape[0], dtype=torch.float64, device=x.device)
    dgu[:, 0::2], dgu[:, 1::2] = dh * u * (s + a * (1 - s)), dh * a
    # the magnitudes that fp32 sums of dh, g and u can be off by 2^-20 of: through g's slope (|.''| < 1) and u
    mg, mu, mh = x.abs() @ wgu[0::2].abs().T, x.abs() @ wgu[1::2].abs().T, dy.abs() @ wd.abs()
    loose = torch.empty_like(dgu)
    loose[:, 0::2] = mh * u.abs() * 1.1 + dh.abs() * (mu * 1.1 + u.abs() * mg)
    loose[:, 1::2] = mh * a.abs() + dh.abs() * mg * 1.1
    hl = mg * 1.1 * u.abs() + a.abs() * mu
    half = torch.finfo(torch.bfloat16).eps / 2
    return ((dgu @ wgu, dgu.T @ x, dy.T @ h),
            lambda hs: ((dgu.abs() * hs + loose * 2.0 ** -20) @ wgu.abs(),
                        (dgu.abs() * hs + loose * 2.0 ** -20).T @ x.abs(),
                        dy.abs().T @ (h.abs() * hs + hl * 2.0 ** -20)))


def check(got, ref, spread, t, terms, what, tokens):
    """Element by element: the operand's rounding (half a step of every term), the
    fp32 sum (2^-20 of the terms' magnitudes: the tensor core's own additions,
    `terms` / 16 of them at 2^-24) and the output's half step; a value below the
    type's smallest normal is off by that type's smallest step at most.  In the
    2-norm two independent roundings, each at most half a step / sqrt(3), stay
    below half a step."""
    import torch
    hs = torch.finfo(t).eps / 2
    tol = ref.abs() * hs + spread * (1 + hs) + torch.finfo(t).tiny * torch.finfo(t).eps
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), (what, float((err / tol).max()))
    if ref.numel() >= 4096:
        assert float(err.norm() / ref.norm()) <= hs, what
        # up to 64 tokens only the output is rounded: half a step / sqrt(3) at most
        if tokens <= 64:
            assert float(err.norm() / ref.norm()) <= 0.6 * hs, what


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("T,H,I", SHAPES)
def test_forward(T, H, I, dtype):
    import torch
    t = getattr(torch, dtype)
    x, wgu, wd, _ = inputs(T, H, I, t)
    y = torch.full_like(x, 9.0)
    ws = torch.empty(q.moe_ffn_workspace_bytes(H, I, T), dtype=torch.uint8, device="cuda")
    q.moe_ffn_forward(wgu, wd, x, y, ws)
    torch.cuda.synchronize()
    assert q.moe_device_status(ws) == 0
    ref, mag = torch_ref(x, wgu, wd)
    # h's rounding and its own fp32 sums (through both factors), then the second sum
    g = x.double().abs() @ wgu.double().abs().T
    gu = x.double() @ wgu.double().T
    hl = (g[:, 0::2] * 1.1 * gu[:, 1::2].abs() + gu[:, 0::2].abs() * g[:, 1::2]) @ wd.double().abs().T
    hs = torch.finfo(t).eps / 2
    tiny = torch.finfo(t).tiny * torch.finfo(t).eps * wd.double().abs().sum(1)
    check(y, ref, mag * (hs + 2.0 ** -20) + hl * 2.0 ** -20 + tiny, t, I, "y", T)


@gpu
@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("T,H,I", SHAPES)
def test_backward(T, H, I, dtype):
    import torch
    t = getattr(torch, dtype)
    x, wgu, wd, dy = inputs(T, H, I, t, seed=1)
    out = [torch.full_like(x, 9.0), torch.full_like(wgu, 9.0), torch.full_like(wd, 9.0)]
    ws = torch.empty(q.moe_ffn_workspace_bytes(H, I, T, backward=True), dtype=torch.uint8, device="cuda")
    q.moe_ffn_backward(wgu, wd, x, dy, ws, dx=out[0], dw_gate_up=out[1], dw_down=out[2])
    torch.cuda.synchronize()
    assert q.moe_device_status(ws) == 0
    refs, spread = torch_ref(x, wgu, wd, dy)
    hs = torch.finfo(t).eps / 2
    least = torch.finfo(t).tiny * torch.finfo(t).eps          # an operand below the normal range
    tiny = (wgu.double().abs().sum(0)[None], x.double().abs().sum(0)[None], dy.double().abs().sum(0)[:, None])
    for got, ref, sp, tn, n, what in zip(out, refs, spread(hs + 2.0 ** -20), tiny, (2 * I, T, T),
                                         ("dx", "dw_gate_up", "dw_down")):
        check(got, ref, sp + tn * least, t, n, what, T)


@gpu
def test_gradient_against_differences():
    """The kernel's gradients along random directions against differences of the 64-bit block."""
    import torch
    x, wgu, wd, dy = inputs(96, 256, 320, torch.bfloat16, seed=2)
    out = [torch.empty_like(v) for v in (x, wgu, wd)]
    ws = torch.empty(q.moe_ffn_workspace_bytes(256, 320, 96, backward=True), dtype=torch.uint8, device="cuda")
    q.moe_ffn_backward(wgu, wd, x, dy, ws, dx=out[0], dw_gate_up=out[1], dw_down=out[2])
    v = [w.double() for w in (x, wgu, wd)]
    for k in range(3):
        d = torch.randn_like(v[k])
        e = 1e-4
        plus, minus = (torch_ref(*[w + (sg * e * d if i == k else 0) for i, w in enumerate(v)])[0] for sg in (1, -1))
        want = ((plus - minus) * dy.double()).sum() / (2 * e)
        # every element is within two half steps, so independent errors add to this; differences are exact to e^2
        noise = (out[k].double() * d).norm() * 2 * 2.0 ** -8
        assert abs(float((out[k].double() * d).sum() - want)) <= 5 * float(noise) + 1e-6 * abs(float(want))


@gpu
def test_outputs_left_out_and_no_tokens():
    import torch
    T, H, I = 70, 192, 136
    x, wgu, wd, dy = inputs(T, H, I, torch.bfloat16, seed=3)
    ws = torch.empty(q.moe_ffn_workspace_bytes(H, I, T, backward=True), dtype=torch.uint8, device="cuda")
    names = ("dx", "dw_gate_up", "dw_down")
    full = {n: torch.empty_like(v) for n, v in zip(names, (x, wgu, wd))}
    q.moe_ffn_backward(wgu, wd, x, dy, ws, **full)
    for mask in range(1, 8):
        part = {n: torch.full_like(full[n], 4.0) for i, n in enumerate(names) if mask >> i & 1}
        q.moe_ffn_backward(wgu, wd, x, dy, ws, **part)
        for n, v in part.items():
            assert torch.equal(v, full[n]), (mask, n)
    empty = {n: torch.full_like(full[n], 4.0) for n in names[1:]}
    q.moe_ffn_backward(wgu, wd, x[:0], dy[:0], ws, dx=x[:0].clone(), **empty)
    assert all(bool((v == 0).all()) for v in empty.values())


@gpu
def test_nothing_outside_the_outputs_and_repeats():
    """Outputs inside larger buffers: the bytes around them stay; the same call gives the same bits."""
    import torch
    T, H, I = 333, 328, 264
    x, wgu, wd, dy = inputs(T, H, I, torch.float16, seed=4)
    ws = torch.empty(q.moe_ffn_workspace_bytes(H, I, T, backward=True), dtype=torch.uint8, device="cuda")
    bufs = [torch.full((v.numel() + 16,), 2.5, dtype=v.dtype, device="cuda") for v in (x, x, wgu, wd)]
    y, dx, dwgu, dwd = (b[8:-8].view(v.shape) for b, v in zip(bufs, (x, x, wgu, wd)))

    def run():
        q.moe_ffn_forward(wgu, wd, x, y, ws)
        q.moe_ffn_backward(wgu, wd, x, dy, ws, dx=dx, dw_gate_up=dwgu, dw_down=dwd)
        return [v.clone() for v in (y, dx, dwgu, dwd)]

    first = run()
    for _ in range(3):
        ws.fill_(255)                                    # nothing is carried over in the workspace
        assert all(torch.equal(a, b) for a, b in zip(first, run()))
    torch.cuda.synchronize()
    assert q.moe_device_status(ws) == 0
    assert all(bool((b[:8] == 2.5).all() and (b[-8:] == 2.5).all()) for b in bufs)


@gpu
@pytest.mark.parametrize("T,H,I", [(40, 256, 192), (900, 1024, 2048)])
def test_captured_step(T, H, I):
    """Forward and backward captured into a graph on a side stream, replayed on new inputs, beside an eager call
    with its own workspace on another stream."""
    import torch
    sets = [inputs(T, H, I, torch.bfloat16, seed=s) for s in (5, 6)]
    mk = lambda: torch.empty(q.moe_ffn_workspace_bytes(H, I, T, backward=True), dtype=torch.uint8, device="cuda")  # noqa: E731

    def outs(s):
        return [torch.empty_like(s[0]), torch.empty_like(s[0]), torch.empty_like(s[1]), torch.empty_like(s[2])]

    def step(s, o, ws, stream=None):
        x, wgu, wd, dy = s
        q.moe_ffn_forward(wgu, wd, x, o[0], ws, stream=stream)
        q.moe_ffn_backward(wgu, wd, x, dy, ws, dx=o[1], dw_gate_up=o[2], dw_down=o[3], stream=stream)

    ws, want = mk(), []
    for s in sets:
        o = outs(s)
        step(s, o, ws)
        want.append(o)
    torch.cuda.synchronize()
    fixed = [v.clone() for v in sets[0]]
    got, other, ws2 = outs(fixed), outs(sets[1]), mk()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        step(fixed, got, ws)
    for k in (1, 0, 1):
        for dst, src in zip(fixed, sets[k]):
            dst.copy_(src)
        torch.cuda.synchronize()
        graph.replay()
        step(sets[1], other, ws2, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[k]))
        assert all(torch.equal(a, b) for a, b in zip(other, want[1]))
    assert q.moe_device_status(ws) == 0 and q.moe_device_status(ws2) == 0


@gpu
def test_infinities_and_nan_stay_in_their_tokens():
    import torch
    T, H, I = 150, 128, 128
    x, wgu, wd, dy = inputs(T, H, I, torch.bfloat16, seed=7)
    ws = torch.empty(q.moe_ffn_workspace_bytes(H, I, T), dtype=torch.uint8, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    q.moe_ffn_forward(wgu, wd, x, y, ws)
    bad = x.clone()
    bad[3, 5], bad[140, 0] = float("nan"), float("inf")
    q.moe_ffn_forward(wgu, wd, bad, z, ws)
    keep = [i for i in range(T) if i not in (3, 140)]
    assert torch.equal(z[keep], y[keep]) and bool(z[3].isnan().all()) and not bool(z[140].isfinite().any())
    # saturated gates: silu'(g) is 0 or 1, nothing overflows on the way
    xs = x * 1000
    out = torch.empty_like(x)
    ws = torch.empty(q.moe_ffn_workspace_bytes(H, I, T, backward=True), dtype=torch.uint8, device="cuda")
    q.moe_ffn_backward(wgu, wd, xs, dy, ws, dx=out)
    ref = torch_ref(xs, wgu, wd, dy)[0][0]
    assert bool(out.isfinite().all()) and float((out.double() - ref).norm() / ref.norm()) <= 2.0 ** -8


@gpu
def test_tune_then_serve():
    """The block as it is used: a training step in 16 bits, the weights packed, the packed block served."""
    import torch
    import moe_inputs as mi
    H, I, T = 256, 128, 24
    x, wgu, wd, dy = inputs(T, H, I, torch.bfloat16, seed=8)
    ws = torch.empty(q.moe_ffn_workspace_bytes(H, I, T, backward=True), dtype=torch.uint8, device="cuda")
    dwgu, dwd = torch.empty_like(wgu), torch.empty_like(wd)
    q.moe_ffn_backward(wgu, wd, x, dy, ws, dw_gate_up=dwgu, dw_down=dwd)
    wgu, wd = wgu - 0.1 * dwgu, wd - 0.1 * dwd
    y = torch.empty_like(x)
    q.moe_ffn_forward(wgu, wd, x, y, ws)
    packed = []
    for w in (wgu, wd):
        codes, scales = mi.gen.quantize_blocks(w.float().cpu().numpy(), 4, 32)
        packed.append((torch.from_numpy(np.ascontiguousarray(codes)).cuda(),
                       torch.from_numpy(np.ascontiguousarray(scales).view(np.int16)).cuda()))
    cfg = q.linear_config_of()
    h, z = torch.empty(T, I, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    q.moe_linear_gated_forward(cfg, *packed[0], x, h)
    q.moe_linear_forward(cfg, *packed[1], h, z)
    # the served block is the 16-bit one on the packed weights
    deq = []
    for (codes, scales), (r, c) in zip(packed, ((2 * I, H), (H, I))):
        d = torch.empty(r, c, device="cuda")
        q.moe_dequant_rows(cfg, codes, scales, 0, r, c, d)
        deq.append(d.double())
    ref, _ = torch_ref(x, *deq)
    assert float((z.double() - ref).norm() / ref.norm()) <= 2.0 ** -8          # two roundings, as above
    exact, _ = torch_ref(x, wgu, wd)
    assert float((y.double() - exact).norm() / exact.norm()) <= 2.0 ** -8
