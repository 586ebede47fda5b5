"""The 8-bit floating-point form on the GPU against its definition in 64 bits:
the quantizers bit for bit, the products within the rounding of their sums.

Tolerance of a product (TOL below): inside a block of 128 the tensor core adds
exact products in fp32, at most 128 additions that each lose up to 2^-23 of the
partial sum (truncation allowed for); the block's two scales are multiplied
(2^-24) and one fused multiply-add per block plus at most 8 additions across a
cluster follow (2^-24 each).  All relative to A = sum |x w| of the output.  Then
one rounding to the output type, eps / 2 of the value."""
import numpy as np
import pytest
import torch

import fp8_util as f8
from post_weight_quantization_05_b200 import _native, api, build_lib

pytestmark = pytest.mark.gpu

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _ready():
    build_lib.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    api.get_status(raise_on_error=False)
    yield
    code, _ = api.get_status(raise_on_error=False)
    assert code == 0


def sum_tol(d):
    return 128 * 2.0 ** -23 + (-(-d // 128) + 9) * 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rand(m, d, seed, dtype=torch.float32, ld=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((m, ld or d), generator=g) * torch.exp(torch.randn((1, ld or d), generator=g))
    return x.to(dtype).cuda()[:, :d]


def bits(codes):
    return codes.contiguous().view(torch.uint8).cpu().numpy()


def quantized_rows(x):
    m, d = x.shape
    c, s = api.fp8_codes(m, d), torch.empty((api.fp8_blocks(d), m), device="cuda")
    api.fp8_quantize_rows(x, c, s)
    return c, s


def quantized_weight(w):
    n, d = w.shape
    c, s = api.fp8_codes(n, d), torch.empty((api.fp8_blocks(n), api.fp8_blocks(d)), device="cuda")
    api.fp8_quantize_weight(w, c, s)
    return c, s


def check_rows(x, c, s):
    want, ws = f8.quantize(x.double().cpu().numpy(), 1)
    assert np.array_equal(s.cpu().numpy(), ws.T)
    assert np.array_equal(bits(c), want)


# ------------------------------------------------------------------ quantizers
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("m,d,ld", [(1, 1, None), (1, 4096, None), (3, 127, None), (9, 128, None), (17, 129, 136),
                                    (8, 1025, 1025), (5, 2309, 2312), (64, 768, 2304), (2, 5000, 5001)])
def test_rows(dtype, m, d, ld):
    x = rand(m, d, 3 * m + d, DTYPES[dtype], ld)
    check_rows(x, *quantized_rows(x))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n,d", [(1, 1), (128, 128), (127, 129), (300, 1000), (256, 4096), (129, 2304)])
def test_weight(dtype, n, d):
    w = rand(n, d, n + d, DTYPES[dtype])
    c, s = quantized_weight(w)
    want, ws = f8.quantize(w.double().cpu().numpy(), 128)
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(bits(c), want)


def test_misaligned_base_and_guard_bytes():
    """A slice that starts off a 16-byte boundary; the bytes behind a row's
    codes and the scales behind the last token stay as they were."""
    x = rand(6, 1000, 5, torch.bfloat16, 1024)[:, 3:900]
    buf = torch.full((6, 1008), 0x5A, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((9, 10), 7.0, device="cuda")
    api.fp8_quantize_rows(x, buf[:, :897], sbuf[:8, :6])
    check_rows(x, buf[:, :897], sbuf[:8, :6])
    assert (buf[:, 897:] == 0x5A).all() and (sbuf[:, 6:] == 7).all() and (sbuf[8] == 7).all()


def test_borders():
    """Quotients on, and one unit in the last place beside, the middle of two
    codes; tiny and huge blocks; zeros of both signs."""
    mid = (f8.TABLE[:126] + f8.TABLE[1:127]) / 2
    rows = []
    for s in (1.0, 0.37, 3.1e-5, 2.0 ** -100, 2.0 ** 100):
        amax = np.float32(448 * s)
        sc = np.float64(np.float32(amax / np.float32(448)))
        t = (mid * sc).astype(np.float32)
        for v in (t, np.nextafter(t, np.float32(np.inf)), np.nextafter(t, np.float32(-np.inf))):
            rows.append(np.concatenate([v, [amax, -0.0]]).astype(np.float32))
            rows.append(-rows[-1])
    rows.append(np.zeros(128, np.float32))
    rows.append(np.full(128, -0.0, np.float32))
    rows.append(np.full(128, 2.0 ** -126, np.float32))
    rows.append(np.full(128, 3.4e38, np.float32))
    x = torch.from_numpy(np.stack(rows)).cuda()
    check_rows(x, *quantized_rows(x))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_every_bf16_ratio(dtype):
    """Every bf16 value down to 2^-20 of the block's largest, for every
    significand of the largest: the quotients next to a middle among them."""
    values = torch.cat([(1 + torch.arange(128) / 128) * 2.0 ** -e for e in range(1, 21)])
    values = torch.cat([values, torch.zeros(-len(values) % 127)]).view(-1, 127)
    values[:, 1::2] *= -1
    tops = 1 + torch.arange(128) / 128
    x = torch.cat([values.expand(128, -1, -1), tops[:, None, None].expand(-1, values.shape[0], 1)], 2)
    x = x.reshape(128, -1).to(DTYPES[dtype]).cuda()
    check_rows(x, *quantized_rows(x))


def test_every_scale():
    """The scale is the correctly rounded amax / 448 for every significand."""
    x = (torch.arange(1 << 23, dtype=torch.int32, device="cuda") + 0x3F800000).view(torch.float32)[:, None]
    c, s = quantized_rows(x)
    assert torch.equal(s[0], x[:, 0] / torch.full_like(x[:, 0], 448.0))
    assert (c.float() == 448).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nonfinite_block(bad):
    x = rand(4, 300, 1)
    x[2, 200] = bad
    c, s = quantized_rows(x)
    code, detail = api.get_status(raise_on_error=False)
    assert (code, detail) == (4, 2)
    assert torch.isnan(s[1, 2]) and torch.isfinite(s).sum() == s.numel() - 1
    assert torch.isnan(c.float()[2, 128:256]).all()
    want, _ = f8.quantize(np.nan_to_num(x[:, :128].double().cpu().numpy()), 1)
    assert np.array_equal(bits(c[:, :128]), want)


# ------------------------------------------------------------------ products
def operands(m, n, d, seed):
    xc, xs = quantized_rows(rand(m, d, seed))
    wc, ws = quantized_weight(rand(n, d, seed + 1) * 0.02)
    return xc, xs, wc, ws


def reference(xc, xs, wc, ws):
    x = f8.values(bits(xc), xs.cpu().numpy().T, 1)
    w = f8.values(bits(wc), ws.cpu().numpy(), 128)
    return x @ w.T, np.abs(x) @ np.abs(w).T


PRODUCTS = [(1, 1, 1), (1, 128, 128), (2, 300, 16), (15, 129, 100), (16, 2304, 768), (17, 640, 129), (33, 257, 2000),
            (64, 128, 4096), (65, 384, 257), (127, 130, 640), (128, 512, 1024), (200, 1000, 333), (513, 700, 896)]


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("m,n,d", PRODUCTS)
def test_product(m, n, d, out):
    ops = operands(m, n, d, m + n + d)
    y = torch.empty((m, n), dtype=DTYPES[out], device="cuda")
    api.fp8_gemm(*ops, y)
    ref, a = reference(*ops)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= sum_tol(d) * a + half_step(y.dtype) * np.abs(ref) + 2.0 ** -25).all()


@pytest.mark.parametrize("out", ["fp32", "bf16", "fp8"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m,n,d", [(1, 128, 128), (3, 300, 1000), (16, 2304, 768), (20, 129, 100), (40, 640, 4096),
                                   (100, 257, 129), (300, 500, 640)])
def test_gated(m, n, d, act, out):
    xc, xs, gc, gs = operands(m, n, d, m + n + d)
    uc, us = quantized_weight(rand(n, d, d) * 0.05)
    g, ag = reference(xc, xs, gc, gs)
    u, au = reference(xc, xs, uc, us)
    h = f8.act(g, act) * u
    # |act'| <= 1.13 for both; 4 roundings of the activation and the product
    # (erfc and exp are within a few units in the last place)
    tol = sum_tol(d) * (1.13 * ag * np.abs(u) + np.abs(f8.act(g, act)) * au) * 1.01 + 16 * 2.0 ** -24 * np.abs(h)
    if out != "fp8":
        y = torch.empty((m, n), dtype=DTYPES[out], device="cuda")
        api.fp8_gated(xc, xs, gc, gs, uc, us, y, act=act)
        err = np.abs(y.double().cpu().numpy() - h)
        assert (err <= tol + half_step(y.dtype) * np.abs(h) + 2.0 ** -25).all()
        return
    y, ys = api.fp8_codes(m, n), torch.empty((api.fp8_blocks(n), m), device="cuda")
    api.fp8_gated(xc, xs, gc, gs, uc, us, y, ys, act=act)
    s = ys.cpu().numpy().T.astype(np.float64)
    amax, worst = f8.block_max(h, 1), f8.block_max(tol, 1)
    assert (np.abs(s - np.maximum(amax, f8.AMAX_FLOOR) / 448) <= worst / 448 + 2.0 ** -24 * s).all()
    # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below 2^-6
    got = f8.values(bits(y), ys.cpu().numpy().T, 1)
    step = np.maximum(2.0 ** -4 * np.abs(got), 2.0 ** -10 * f8.spread(s, 1, m, n))
    assert (np.abs(got - h) <= tol + 1.001 * step).all()


def test_same_bits_and_columns_do_not_mix():
    """The same call twice gives the same bits, and a token's outputs do not
    depend on how many others it came with."""
    ops = operands(40, 700, 1500, 9)
    y = [torch.empty((40, 700), device="cuda") for _ in range(2)]
    for t in y:
        api.fp8_gemm(*ops, t)
    assert torch.equal(y[0], y[1])
    xc, xs, wc, ws = ops
    one = torch.empty((1, 700), device="cuda")
    api.fp8_gemm(xc[7:8], xs[:, 7:8], wc, ws, one)
    ref, a = reference(*ops)
    assert (np.abs(one.double().cpu().numpy()[0] - ref[7]) <= sum_tol(1500) * a[7]).all()


def test_pitched_and_untouched():
    """Slices of wider buffers on every side; the columns and rows around the
    output stay as they were."""
    m, n, d = 37, 301, 500
    xc, xs, wc, ws = operands(m + 5, n, d, 4)
    wide = torch.full((m + 2, n + 13), 9.0, device="cuda")
    y = wide[1:m + 1, 5:5 + n]
    api.fp8_gemm(xc[3:m + 3], xs[:, 3:m + 3], wc, ws, y)
    ref, a = reference(xc[3:m + 3], xs[:, 3:m + 3], wc, ws)
    assert (np.abs(y.double().cpu().numpy() - ref) <= sum_tol(d) * a + 2.0 ** -24 * np.abs(ref)).all()
    assert (wide[0] == 9).all() and (wide[-1] == 9).all() and (wide[:, :5] == 9).all() and (wide[:, 5 + n:] == 9).all()


def test_gated_codes_leave_the_padding():
    m, n, d = 21, 200, 256
    xc, xs, gc, gs = operands(m, n, d, 2)
    buf = torch.full((m, 224), 0x33, dtype=torch.uint8, device="cuda")
    ys = torch.full((3, 30), 5.0, device="cuda")
    api.fp8_gated(xc, xs, gc, gs, gc, gs, buf[:, :n], ys[:2, :m])
    assert (buf[:, n:] == 0x33).all() and (ys[:, m:] == 5).all() and (ys[2] == 5).all()


def test_nan_scale_reaches_its_token_only():
    ops = operands(5, 200, 300, 8)
    ops[1][1, 3] = float("nan")
    y = torch.empty((5, 200), device="cuda")
    api.fp8_gemm(*ops, y)
    assert torch.isnan(y[3]).all() and torch.isfinite(y[[0, 1, 2, 4]]).all()


def test_layer_runs_through():
    """A gated feed-forward layer as it is served: quantize, the gated pair to
    codes, the down projection.  Captured into a graph and replayed on new inputs."""
    m, d, f = 24, 512, 1280
    gate, up, down = (quantized_weight(rand(*s, i) * 0.02) for i, s in enumerate([(f, d), (f, d), (d, f)]))
    x = rand(m, d, 77, torch.bfloat16).contiguous()
    xc, xs = api.fp8_codes(m, d), torch.empty((api.fp8_blocks(d), m), device="cuda")
    hc, hs = api.fp8_codes(m, f), torch.empty((api.fp8_blocks(f), m), device="cuda")
    y = torch.empty((m, d), dtype=torch.bfloat16, device="cuda")

    def layer():
        api.fp8_quantize_rows(x, xc, xs)
        api.fp8_gated(xc, xs, *gate, *up, hc, hs)
        api.fp8_gemm(hc, hs, *down, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
    torch.cuda.current_stream().wait_stream(side)
    first = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    x.copy_(rand(m, d, 78, torch.bfloat16))
    graph.replay()
    replayed = y.clone()
    layer()
    assert torch.equal(replayed, y) and not torch.equal(first, y)
    x.copy_(rand(m, d, 77, torch.bfloat16))
    graph.replay()
    assert torch.equal(first, y)
    wide = [f8.values(bits(c), s.cpu().numpy(), 128) for c, s in (gate, up, down)]
    xv = x.double().cpu().numpy()
    h = f8.act(xv @ wide[0].T, "silu") * (xv @ wide[1].T)
    ref = h @ wide[2].T
    # two e4m3 quantizations of independent rounding errors, 2^-4 at most each
    err = np.linalg.norm(y.double().cpu().numpy() - ref) / np.linalg.norm(ref)
    assert err <= 2 * 2.0 ** -4


# Every form a product of more than 32 tokens has: one, two or four SM pairs per
# tile, tiles of 128 and 256 weight rows, several rounds of tiles per pair.
@pytest.mark.parametrize("m,n,d", [(40, 300, 10000), (100, 4096, 4096), (512, 4096, 1000), (100, 8192, 4000),
                                   (300, 11008, 256), (1100, 5000, 700), (100, 8192, 8000), (2300, 4096, 2000)])
def test_product_forms(m, n, d):
    ops = operands(m, n, d, m + d)
    y = torch.empty((m, n), device="cuda")
    api.fp8_gemm(*ops, y)
    ref, a = reference(*ops)
    assert (np.abs(y.double().cpu().numpy() - ref) <= sum_tol(d) * a + 2.0 ** -24 * np.abs(ref)).all()


@pytest.mark.parametrize("out", ["fp16", "fp8"])
@pytest.mark.parametrize("m,n,d", [(40, 1000, 5000), (40, 2900, 5000), (300, 11008, 256), (1100, 3000, 700)])
def test_gated_forms(m, n, d, out):
    test_gated(m, n, d, "silu", out)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m", [1, 20, 70])
def test_gates_near_the_largest_number(m, act):
    """Gates past 2^127: the activation is the gate itself, or nothing."""
    one = torch.full((128, 128), 0x38, dtype=torch.uint8, device="cuda")      # 1.0
    x = torch.zeros((m, 128), dtype=torch.uint8, device="cuda")
    x[:, 0] = torch.where(torch.arange(m, device="cuda") % 2 == 0, 0x38, 0xB8).byte()
    xs = torch.ones((1, m), device="cuda")
    y = torch.empty((m, 128), device="cuda")
    api.fp8_gated(x, xs, one, torch.full((1, 1), 3e38, device="cuda"), one, torch.full((1, 1), 2.0 ** -100, device="cuda"),
                  y, act=act)
    want = float(np.float32(3e38)) * 2.0 ** -100
    got = y.double().cpu().numpy()
    assert (np.abs(got[::2] - want) <= 16 * 2.0 ** -24 * want).all() and (got[1::2] == 0).all()


@pytest.mark.parametrize("m", [5, 37, 301])
def test_scales_behind_the_last_token(m):
    """Token scales in rows that reach past the last token, aligned and not: what
    lies there is another caller's."""
    n, d = 300, 700
    xc, xs, wc, ws = operands(m, n, d, m)
    ref, a = reference(xc, xs, wc, ws)
    for pitch, off in ((-(-m // 4) * 4 + 4, 0), (m + 6, 1), (-(-m // 4) * 4 + 4, 4)):
        room = torch.full((xs.shape[0], pitch + off), float("nan"), device="cuda")
        wide = room[:, off:off + m]
        wide.copy_(xs)
        y = torch.empty((m, n), device="cuda")
        api.fp8_gemm(xc, wide, wc, ws, y)
        assert (np.abs(y.double().cpu().numpy() - ref) <= sum_tol(d) * a + 2.0 ** -24 * np.abs(ref)).all()


def test_calls_on_two_streams_at_once():
    """Products of every shape on two streams, interleaved: each as by itself."""
    shapes = [(1, 2048, 4096), (24, 1024, 4096), (100, 4096, 4096), (512, 4096, 1000), (300, 2048, 256)]
    ops = [operands(m, n, d, m) for m, n, d in shapes]
    alone = []
    for o, (m, n, d) in zip(ops, shapes):
        alone.append(torch.empty((m, n), device="cuda"))
        api.fp8_gemm(*o, alone[-1])
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [[torch.full_like(y, float("nan")) for y in alone] for _ in streams]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, ys, order in zip(streams, both, (1, -1)):
            for i in range(len(shapes))[::order]:
                api.fp8_gemm(*ops[i], ys[i], stream=s)
    torch.cuda.synchronize()
    for ys in both:
        assert all(torch.equal(a, b) for a, b in zip(alone, ys))


def test_refusals():
    x, w = rand(4, 256, 1), rand(128, 256, 2)
    c, s = quantized_rows(x)
    wc, ws = quantized_weight(w)
    y = torch.empty((4, 128), device="cuda")
    with pytest.raises(ValueError):
        api.fp8_quantize_rows(x.double(), c, s)
    with pytest.raises(ValueError):
        api.fp8_quantize_rows(x, c[:, :128], s)
    with pytest.raises(ValueError):
        api.fp8_quantize_rows(x, c, s[:1])
    with pytest.raises(api.GPTQError):
        api.fp8_quantize_rows(x[:, :100], torch.empty((4, 100), dtype=torch.uint8, device="cuda"), s[:1])   # pitch
    with pytest.raises(ValueError):
        api.fp8_gemm(c, s, wc, ws, y[:, :100])
    with pytest.raises(ValueError):
        api.fp8_gemm(c, s, wc, ws.t(), y)
    with pytest.raises(ValueError):
        api.fp8_gemm(c.cpu(), s, wc, ws, y)
    with pytest.raises(ValueError):
        api.fp8_gated(c, s, wc, ws, wc, ws, y, act="relu")
    with pytest.raises(ValueError):
        api.fp8_gated(c, s, wc, ws, wc, ws, api.fp8_codes(4, 128))
    with pytest.raises(ValueError):
        api.fp8_gated(c, s, wc, ws, wc, ws, y, s)
    api.fp8_gemm(c[:0], s[:, :0], wc, ws, y[:0])                 # no tokens: nothing to do
    assert _native.load().gptq_get_status(None, None) == 0
