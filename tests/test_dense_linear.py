"""Products with one packed matrix (moe_linear_forward) and the gated pair of
projections (moe_linear_gated_forward) against the definition in 64 bits."""
import ctypes

import numpy as np
import pytest

import quantized_expert_ffn_moe_b200 as q
from quantized_expert_ffn_moe_b200 import build as qbuild

FORMATS = {"h32": dict(block=32), "h128": dict(block=128), "h32half": dict(block=32, half_levels=True),
           "h128half": dict(block=128, half_levels=True), "e32": dict(block=32, fp8_scales=True)}


# ------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return q.load_library()


A = 1 << 20          # never dereferenced: every call below is refused


def linear(lib, cfg, codes=A, scales=2 * A, rs=None, rows=64, cols=256, bias=None, x=3 * A, xt=q.MOE_BF16, T=4, y=4 * A,
           yt=q.MOE_BF16):
    return lib.moe_linear_forward(cfg and ctypes.byref(cfg), codes, scales, rs, rows, cols, bias, x, xt, T, y, yt, None)


def gated(lib, cfg, codes=A, scales=2 * A, rs=None, inter=64, cols=256, x=3 * A, xt=q.MOE_BF16, T=4, h=4 * A,
          ht=q.MOE_BF16):
    return lib.moe_linear_gated_forward(cfg and ctypes.byref(cfg), codes, scales, rs, inter, cols, x, xt, T, h, ht, None)


@pytest.mark.parametrize("call", [linear, gated])
def test_refusals(lib, call):
    c = q.linear_config_of()
    out, ot = ("y", "yt") if call is linear else ("h", "ht")
    n = "rows" if call is linear else "inter"
    invalid, unsupported = -1, -2
    assert call(lib, None) == invalid
    for name in ("codes", "scales", "x", out):
        assert call(lib, c, **{name: None}) == invalid
        assert call(lib, c, **{name: 5 * A + 8}) == invalid
    for kw in ({n: 0}, {n: -1}, {"cols": 0}, {"T": -1}, {"xt": q.MOE_FP32}, {"xt": 7}, {ot: 3}, {ot: -1}):
        assert call(lib, c, **kw) == invalid, kw
    assert call(lib, c, rs=5 * A) == invalid                      # fp16 scales take no row scales
    c8 = q.linear_config_of(fp8_scales=True)
    assert call(lib, c8) == invalid                               # fp8 scales need them
    assert call(lib, c8, rs=5 * A + 4) == invalid
    for bad in (dict(bits=2, block=16), dict(block=64), dict(block=16), dict(bits=3), dict(block=128, fp8_scales=True),
                dict(half_levels=True, fp8_scales=True)):
        assert call(lib, q.linear_config_of(**bad), rs=5 * A) == unsupported, bad
    for kw in ({"cols": 48}, {"cols": 32768 + 32}, {n: (1 << 30) + 1}):
        assert call(lib, c, **kw) == unsupported, kw
    assert call(lib, q.linear_config_of(block=128), cols=160) == unsupported
    # x [4][256] and the output overlap from either side
    assert call(lib, c, **{out: 3 * A + 4 * 256 * 2 - 16}) == invalid
    assert call(lib, c, **{out: 3 * A - 16}) == invalid
    # no tokens: nothing is launched, no pointer is looked at
    assert call(lib, c, T=0, x=None, codes=None) == 0
    if call is linear:
        assert linear(lib, c, bias=5 * A + 2) == invalid
    assert lib.moe_linear_device_status(None) == invalid


def test_binding_refusals(lib):
    torch = pytest.importorskip("torch")
    c = q.linear_config_of()
    codes, scales = torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(64, 8, dtype=torch.float16)
    x, y = torch.zeros(2, 256, dtype=torch.bfloat16), torch.zeros(2, 64, dtype=torch.bfloat16)
    for kw in (dict(x=x.float()), dict(x=torch.zeros(256, 2, dtype=torch.bfloat16).T), dict(y=y[:1]),
               dict(codes=codes[:63]), dict(scales=scales[:, :4].contiguous()), dict(y=y.double()),
               dict(bias=torch.zeros(63)), dict(bias=torch.zeros(64, dtype=torch.float16)), dict()):
        a = {"codes": codes, "scales": scales, "x": x, "y": y, "bias": None, **kw}
        with pytest.raises(ValueError):       # the last one: tensors of the host
            q.moe_linear_forward(c, a["codes"], a["scales"], a["x"], a["y"], bias=a["bias"])
    with pytest.raises(ValueError):
        q.moe_linear_gated_forward(c, codes, scales, x, y)          # 64 outputs need 128 rows
    with pytest.raises(q.MoeError):
        q.moe_linear_forward(q.linear_config_of(block=96), codes, scales, x, y)


# ------------------------------------------------------------ on the GPU
gpu = pytest.mark.gpu


def matrix(rows, cols, block=32, half_levels=False, fp8_scales=False, seed=0):
    """Random codes and scales, all 16 codes in use, on the device; the weights in 64 bits on the host."""
    import torch
    r = np.random.default_rng(seed)
    codes = r.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
    nb = cols // block
    if fp8_scales:
        sb = r.integers(1, 0x7e, (rows, nb)).astype(np.uint8) | (r.integers(0, 2, (rows, nb)).astype(np.uint8) << 7)
        rs = (np.exp(r.normal(size=rows)) * 1e-4).astype(np.float32)
        e, m = (sb >> 3) & 15, (sb & 7).astype(np.float64)
        s = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.astype(np.float64) - 7)) * np.where(sb >> 7, -1.0, 1.0)
        s = s * rs.astype(np.float64)[:, None]
    else:
        sb = (r.normal(size=(rows, nb)) * 0.01).astype(np.float16)
        rs, s = None, sb.astype(np.float64)
    c = np.empty((rows, cols))
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    off = 7.5 if half_levels else 8.0
    w = ((c - off).reshape(rows, nb, block) * s[:, :, None]).reshape(rows, cols)
    # what an element can contribute before its offset is taken off: bounds the rounding of the sums
    big = ((c + off).reshape(rows, nb, block) * np.abs(s)[:, :, None]).reshape(rows, cols)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    return dev(codes), dev(sb), dev(rs), w, big


def tokens(T, cols, dtype, seed=1):
    import torch
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, cols, generator=g).to(dtype).cuda()


def bound(x, big, cols, out=None):
    """How far fp32 sums may be off: a block's start and its two products of 16
    terms round four times at most at 2^-23 of the magnitudes that meet there,
    and the cols / 32 scaled block sums add with 2^-24 each; the activations'
    own bound 2^-35 of the row's largest is counted for every column.  Batches
    of more than 8 tokens with results of 16 bits (`out`) take each weight
    rounded to fp16 once, half a step of every term (E4M3 weights are exact)."""
    X = np.abs(x)
    mag = X @ big.T
    tiny = X.max(1, keepdims=True) * big.sum(1)[None] * 2.0 ** -35
    weights = 2.0 ** -11 if out is not None and out.itemsize == 2 and len(x) > 8 else 0.0
    return mag * (weights + 2.0 ** -21 + (cols / 32 + 20) * 2.0 ** -24) + tiny


def half_step(t):
    import torch
    return torch.finfo(t).eps / 2


CASES = [
    # T, rows, cols: every token group size, ragged rows, one block, columns off the stage and the copy width
    (1, 1, 32), (1, 16, 64), (2, 17, 96), (3, 15, 128), (5, 33, 160), (8, 256, 256), (1, 2048, 2048), (7, 100, 2080),
    (9, 48, 1056), (16, 130, 4096), (17, 64, 4128), (32, 31, 2048), (33, 50, 512), (64, 77, 8192), (100, 40, 1024), (48, 300, 544), (10, 700, 4096), (16, 150000, 128), (12, 40, 32), (1000, 64, 512), (64, 20481, 1056),
    (3, 40001, 1056), (8, 30000, 2048), (1, 50000, 512),
    (1, 3000, 768), (4, 40, 32768),
]


@gpu
@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("T,rows,cols", CASES)
def test_linear(T, rows, cols, fmt):
    import torch
    f = FORMATS[fmt]
    if cols % f["block"]:
        cols += 128 - cols % 128
    codes, scales, rs, w, big = matrix(rows, cols, **f)
    cfg = q.linear_config_of(**f)
    for xt, yt, bias in ((torch.bfloat16, torch.bfloat16, False), (torch.float16, torch.float32, True),
                         (torch.float16, torch.float16, True)):
        x = tokens(T, cols, xt)
        b = torch.randn(rows, generator=torch.Generator().manual_seed(3)).cuda() if bias else None
        y = torch.full((T, rows), 7.0, dtype=yt, device="cuda")
        q.moe_linear_forward(cfg, codes, scales, x, y, row_scales=rs, bias=b)
        xd = x.double().cpu().numpy()
        ref = xd @ w.T
        if bias:
            ref = ref + b.double().cpu().numpy()
        err = np.abs(y.double().cpu().numpy() - ref)
        # + 2^-22: the powers of two are exact; the row scale and the bias round once each
        tol = np.abs(ref) * (half_step(yt) + 2.0 ** -22) + bound(xd, big, cols, yt)
        assert (err <= tol).all(), (xt, yt, float((err / tol).max()))


@gpu
@pytest.mark.parametrize("fmt", sorted(FORMATS))
@pytest.mark.parametrize("T,inter,cols", [(1, 1, 32), (1, 768, 2048), (3, 7, 128), (8, 8, 256), (11, 50, 1056),
                                          (20, 129, 2048), (64, 24, 512)])
def test_gated(T, inter, cols, fmt):
    import torch
    f = FORMATS[fmt]
    if cols % f["block"]:
        cols += 128 - cols % 128
    codes, scales, rs, w, big = matrix(2 * inter, cols, seed=5, **f)
    for xt, ht in ((torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16), (torch.bfloat16, torch.float32)):
        x = tokens(T, cols, xt) * 0.25
        h = torch.empty(T, inter, dtype=ht, device="cuda")
        q.moe_linear_gated_forward(q.linear_config_of(**f), codes, scales, x, h, row_scales=rs)
        xd = x.double().cpu().numpy()
        z, dz = xd @ w.T, bound(xd, big, cols, ht) + np.abs(xd @ w.T) * 2.0 ** -22
        g, u, dg, du = z[:, 0::2], z[:, 1::2], dz[:, 0::2], dz[:, 1::2]
        a = g / (1 + np.exp(-g))
        # |silu'| < 1.1; exp, the division and the product round in fp32
        tol = (np.abs(u) + du) * 1.1 * dg + np.abs(a) * du + np.abs(a * u) * (half_step(ht) + 2.0 ** -20) + 2.0 ** -24
        err = np.abs(h.double().cpu().numpy() - a * u)
        assert (err <= tol).all(), (xt, ht, float((err / tol).max()))


@gpu
def test_agrees_with_the_dequantizer():
    """Unit vectors read single weights: exactly what moe_dequant_rows writes."""
    import torch
    for f in FORMATS.values():
        codes, scales, rs, w, _ = matrix(37, 256, seed=8, **f)
        cfg = q.linear_config_of(**f)
        x = torch.eye(256, dtype=torch.bfloat16, device="cuda")[::5].contiguous()
        y = torch.empty(x.shape[0], 37, device="cuda")
        q.moe_linear_forward(cfg, codes, scales, x, y, row_scales=rs)
        d = torch.empty(37, 256, device="cuda")
        q.moe_dequant_rows_scaled(cfg, codes, scales, rs, 0, 37, 256, d)
        assert torch.equal(y, d.T[::5])


@gpu
@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** -100, 1.0])
@pytest.mark.parametrize("T,out", [(6, "float32"), (30, "float32"), (30, "bfloat16")])
def test_extreme_activations(scale, T, out):
    """Rows of very large, very small, zero and mixed magnitudes; infinities and NaN stay in their rows."""
    import torch
    cols, yt = 512, getattr(torch, out)
    codes, scales, rs, w, big = matrix(24, cols, seed=9)
    x = tokens(T, cols, torch.float32, seed=4).cpu()
    x[1] = 0
    x[2] *= 2.0 ** -torch.arange(cols).remainder(24)          # elements far below the row's largest
    x[3, 5], x[4, 7] = float("inf"), float("nan")
    xb = (x * scale).to(torch.bfloat16).cuda()
    y = torch.empty(T, 24, dtype=yt, device="cuda")
    q.moe_linear_forward(q.linear_config_of(), codes, scales, xb, y)
    got, xd = y.double().cpu().numpy(), xb.double().cpu().numpy()
    assert np.isnan(got[3:5]).all() and (got[1] == 0).all()
    keep = [r for r in range(T) if r not in (3, 4)]
    with np.errstate(invalid="ignore"):
        tol = np.abs(xd @ w.T) * (half_step(yt) + 2.0 ** -22) + bound(xd, big, cols, yt)
        err = np.abs(got - xd @ w.T)
    assert (err[keep] <= tol[keep]).all()


@gpu
@pytest.mark.parametrize("T,out", [(3, "float32"), (40, "float32"), (40, "bfloat16")])
def test_zero_scales_and_extreme_scales(T, out):
    import torch
    cols, yt = 384, getattr(torch, out)
    codes, scales, rs, w, big = matrix(20, cols, seed=10)
    scales[3] = 0
    scales[4, ::2] = 65504.0
    scales[5] = 2.0 ** -24
    s = scales.double().cpu().numpy()
    c = np.empty((20, cols))
    raw = codes.cpu().numpy()
    c[:, 0::2], c[:, 1::2] = raw & 15, raw >> 4
    w = ((c - 8).reshape(20, -1, 32) * s[:, :, None]).reshape(20, cols)
    big = ((c + 8).reshape(20, -1, 32) * np.abs(s)[:, :, None]).reshape(20, cols)
    x = tokens(T, cols, torch.float16)
    y = torch.empty(T, 20, dtype=yt, device="cuda")
    q.moe_linear_forward(q.linear_config_of(), codes, scales, x, y)
    xd = x.double().cpu().numpy()
    ref = xd @ w.T
    err = np.abs(y.double().cpu().numpy() - ref)
    # a row's blocks whose scale is far below its largest: fp16's least step under the row's power of two, 2^-34 of
    # that largest scale, for each of a block's 32 levels of at most 8
    least = np.abs(xd).sum(1, keepdims=True) * np.abs(s).max(1)[None] * 2.0 ** -34
    assert (err <= np.abs(ref) * (half_step(yt) + 2.0 ** -22) + bound(xd, big, cols, yt) + least).all()
    assert (y[:, 3] == 0).all()


@gpu
@pytest.mark.parametrize("T,rows,cols", [(40, 777, 2048), (4, 777, 2048), (16, 4097, 8192), (64, 1025, 4128)])
@pytest.mark.parametrize("out", ["bfloat16", "float32"])
def test_repeats_and_stays_inside_its_output(T, rows, cols, out):
    """The same call gives the same bits, and nothing is written outside y."""
    import torch
    yt = getattr(torch, out)
    codes, scales, rs, _, _ = matrix(rows, cols, seed=11)
    cfg = q.linear_config_of()
    x = tokens(T, cols, torch.bfloat16)
    flat = torch.full((T * rows + 16,), 3.5, dtype=yt, device="cuda")
    y = flat[8:8 + T * rows].view(T, rows)                    # 16-byte aligned inside the guard
    q.moe_linear_forward(cfg, codes, scales, x, y)
    first = y.clone()
    for _ in range(5):
        y.zero_()
        q.moe_linear_forward(cfg, codes, scales, x, y)
        assert torch.equal(first, y)
    assert (flat[:8] == 3.5).all() and (flat[8 + T * rows:] == 3.5).all()
    assert q.moe_linear_device_status() == 0


@gpu
@pytest.mark.parametrize("T,rows,cols,out", [(4, 512, 1024, "bfloat16"), (16, 2050, 8192, "bfloat16"),
                                             (16, 2050, 8192, "float32"), (64, 8192, 4096, "bfloat16")])
def test_streams_and_graphs(T, rows, cols, out):
    """Two streams at once, and a captured call replayed on new inputs."""
    import torch
    yt = getattr(torch, out)
    codes, scales, rs, _, _ = matrix(rows, cols, seed=12)
    cfg = q.linear_config_of()
    xs = [tokens(T, cols, torch.bfloat16, seed=s) for s in range(2)]
    want = []
    for x in xs:
        y = torch.empty(T, rows, dtype=yt, device="cuda")
        q.moe_linear_forward(cfg, codes, scales, x, y)
        want.append(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [torch.empty_like(want[0]) for _ in xs]
    for _ in range(20):
        for s, x, y in zip(streams, xs, got):
            q.moe_linear_forward(cfg, codes, scales, x, y, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, y = xs[0].clone(), torch.empty_like(want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):                                   # each waits for the one before it
            q.moe_linear_forward(cfg, codes, scales, x, y)
    for k in (1, 0):
        x.copy_(xs[k])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k])
    assert q.moe_linear_device_status() == 0


@gpu
@pytest.mark.parametrize("T,H,I", [(5, 512, 384), (48, 2048, 4096)])
def test_packed_block_serves(T, H, I):
    """Gate/up then down, as a dense block is served: against the definition in 64 bits."""
    import torch
    cgu, sgu, _, wgu, _ = matrix(2 * I, H, seed=13)
    cd, sd, _, wd, _ = matrix(H, I, seed=14)
    cfg = q.linear_config_of()
    x = tokens(T, H, torch.bfloat16)
    h = torch.empty(T, I, dtype=torch.float16, device="cuda")
    y = torch.empty(T, H, device="cuda")
    for _ in range(3):                       # back to back: the second call waits for the first one's h
        h.zero_()
        q.moe_linear_gated_forward(cfg, cgu, sgu, x, h)
        q.moe_linear_forward(cfg, cd, sd, h, y)
    xd = x.double().cpu().numpy()
    z = xd @ wgu.T
    hid = z[:, 0::2] / (1 + np.exp(-z[:, 0::2])) * z[:, 1::2]
    ref = hid @ wd.T
    # h rounds to fp16 (2^-11 of each element, and 2^-25 below its smallest step), with more than 8 tokens after its
    # weights did (2^-11 of every term, through both factors); the rest is fp32
    dh = np.abs(hid) * 2.0 ** -11 + 2.0 ** -25
    if T > 8:
        m = np.abs(xd) @ np.abs(wgu).T * 2.0 ** -11
        g, u = z[:, 0::2], z[:, 1::2]
        dh = dh + (np.abs(u) + m[:, 1::2]) * 1.1 * m[:, 0::2] + np.abs(g) * m[:, 1::2]
    tol = dh @ np.abs(wd).T * 1.01 + np.abs(ref) * 2.0 ** -18
    assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()
