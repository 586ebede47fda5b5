"""The gated pair's codes against the quantizer's, bit for bit, in every form of
the product; more blocks of k than the kernels keep scales for; arrays whose
elements lie further apart than 32 bits can count."""
import numpy as np
import pytest
import torch

import fp8_util as f8
from post_weight_quantization_05_b200 import api, build_lib
from test_gpu_fp8 import bits, check_rows, operands, quantized_rows, quantized_weight, rand, reference, sum_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    build_lib.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    api.get_status(raise_on_error=False)
    yield
    code, _ = api.get_status(raise_on_error=False)
    assert code == 0


# up to 16 and up to 32 tokens; SM pairs by four, two and one per tile; several rounds of tiles
GATED = [(1, 300, 1000), (16, 2304, 768), (32, 129, 700), (40, 1000, 5000), (40, 2900, 5000), (300, 11008, 256),
         (1100, 3000, 700)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m,n,d", GATED)
def test_codes_are_those_of_the_values(m, n, d, act):
    xc, xs, gc, gs = operands(m, n, d, m + n + d)
    uc, us = quantized_weight(rand(n, d, d) * 0.05)
    h = torch.empty((m, n), device="cuda")
    y, ys = api.fp8_codes(m, n), torch.empty((api.fp8_blocks(n), m), device="cuda")
    api.fp8_gated(xc, xs, gc, gs, uc, us, h, act=act)
    api.fp8_gated(xc, xs, gc, gs, uc, us, y, ys, act=act)
    want, ws = quantized_rows(h)
    assert torch.equal(ys, ws) and np.array_equal(bits(y), bits(want))
    again, zs = api.fp8_codes(m, n), torch.empty_like(ys)
    api.fp8_gated(xc, xs, gc, gs, uc, us, again, zs, act=act)
    assert torch.equal(zs, ys) and np.array_equal(bits(again), bits(y))


@pytest.mark.parametrize("m,n,d", GATED[3:])
def test_gelu_forms(m, n, d):
    from test_gpu_fp8 import test_gated
    test_gated(m, n, d, "gelu", "fp16")


# many more blocks of k than either kernel keeps scales for, in one tile and over several
@pytest.mark.parametrize("m,n,d", [(1, 300, 30000), (20, 300, 30000), (40, 300, 30000), (300, 700, 20000),
                                   (1100, 5000, 3000)])
def test_scales_of_many_blocks(m, n, d):
    """Every block's own scales, whichever of the kernel's warps is ahead: near
    the definition, and the same bits on every call."""
    ops = operands(m, n, d, m)
    y = [torch.empty((m, n), device="cuda") for _ in range(2)]
    for _ in range(5):
        for t in y:
            api.fp8_gemm(*ops, t)
        assert torch.equal(y[0], y[1])
    ref, a = reference(*ops)
    assert (np.abs(y[0].double().cpu().numpy() - ref) <= sum_tol(d) * a + 2.0 ** -24 * np.abs(ref)).all()


def apart(src, pitch):
    """A copy of src [rows, cols] whose rows lie `pitch` elements apart."""
    rows, cols = src.shape
    buf = torch.empty(((rows - 1) * pitch + cols,), dtype=src.dtype, device="cuda")
    out = buf.as_strided((rows, cols), (pitch, 1))
    out.copy_(src)
    return out


@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 1000), (torch.float32, 300)])
def test_quantizers_past_32_bits(dtype, d):
    far = 1 << 30                                         # the fifth row lies 2^32 elements behind the first
    x = rand(5, d, 6, dtype)
    c = apart(torch.zeros((5, d), dtype=torch.uint8, device="cuda"), far)
    s = apart(torch.zeros((api.fp8_blocks(d), 5), device="cuda"), far)
    api.fp8_quantize_rows(apart(x, far), c, s)
    check_rows(x, c, s)
    c = apart(torch.zeros((5, d), dtype=torch.uint8, device="cuda"), far)
    s = torch.zeros((1, api.fp8_blocks(d)), device="cuda")
    api.fp8_quantize_weight(apart(x, far), c, s)
    want, ws = f8.quantize(x.double().cpu().numpy(), 128)
    assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(bits(c), want)


@pytest.mark.parametrize("m", [20, 70])
def test_products_past_32_bits(m):
    n, d = 150, 300
    xc, xs, wc, ws = operands(m, n, d, m)
    far = (1 << 32) // (m - 1) // 16 * 16 + 16            # the last row lies past 2^32 elements
    x, w = apart(xc.view(torch.uint8), far), apart(wc.view(torch.uint8), (1 << 32) // (n - 1) // 16 * 16 + 16)
    scales = apart(xs, 1 << 31)                           # and the last block's scales
    y = apart(torch.zeros((m, n), dtype=torch.bfloat16, device="cuda"), far)
    api.fp8_gemm(x, scales, w, ws, y)
    ref, a = reference(xc, xs, wc, ws)
    tol = sum_tol(d) * a + 2.0 ** -8 * np.abs(ref) + 2.0 ** -25
    assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()
    values, codes = torch.empty((m, n), device="cuda"), apart(torch.zeros((m, n), dtype=torch.uint8, device="cuda"), far)
    ys = apart(torch.zeros((2, m), device="cuda"), 1 << 32)
    api.fp8_gated(x, scales, w, ws, w, ws, values)
    api.fp8_gated(x, scales, w, ws, w, ws, codes, ys)
    want, qs = quantized_rows(values)
    assert torch.equal(ys.contiguous(), qs) and np.array_equal(bits(codes), bits(want))
