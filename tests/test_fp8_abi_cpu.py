"""CPU-only checks of the 8-bit floating-point calls and the token scores: bad
arguments are refused on the host before any CUDA call, empty calls succeed, and
the tests' own 64-bit forms agree with torch's e4m3 conversion."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_util as f8
from post_weight_quantization_05_b200 import _native, build_lib

P = ctypes.c_void_p
BAD, UNALIGNED = 1, P(0x10000004)
X, C, S, W, U, V, Y, T = (P(0x10000000 * (i + 1)) for i in range(8))   # far apart, 16-byte aligned, never read


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return _native.load()


def refused(fn, good, changes):
    """Every change of the good arguments (by position) is refused."""
    for at, value in changes:
        args = list(good)
        args[at] = value
        assert fn(*args) == BAD, (at, value)


def test_quantize_rows_refusals(lib):
    #       x  dtype m  d    ldx  codes ldc  scales lds stream
    good = (X, 1, 4, 300, 300, C, 304, S, 4, None)
    refused(lib.gptq_fp8_quantize_rows, good, [
        (0, None), (0, P(0x10000001)), (1, 3), (1, -1), (2, -1), (2, 1 << 25), (3, 0), (3, 1 << 19), (4, 299),
        (4, 1 << 40), (5, None), (5, P(0x20000008)), (6, 300), (6, 288), (7, None), (7, P(0x30000002)), (8, 3),
        (5, P(X.value + 16)), (7, P(X.value + 16)), (7, P(C.value + 16))])
    assert lib.gptq_fp8_quantize_rows(None, 1, 0, 300, 300, None, 304, None, 0, None) == 0


def test_quantize_weight_refusals(lib):
    good = (X, 0, 200, 300, 300, C, 304, S, None)
    refused(lib.gptq_fp8_quantize_weight, good, [
        (0, None), (0, P(0x10000002)), (1, 3), (2, 0), (2, 1 << 23), (3, 0), (3, 1 << 19), (4, 299), (5, None),
        (5, P(0x20000004)), (6, 299), (6, 312), (7, None), (7, P(0x30000002)), (5, X), (7, X), (7, C)])


def test_product_refusals(lib):
    #       x  ldx  xs lds w  ldw  ws m  n    d    out y  ldy
    good = (X, 304, S, 8, W, 304, U, 8, 200, 300, 0, Y, 200, None)
    refused(lib.gptq_fp8_gemm, good, [
        (0, None), (0, UNALIGNED), (1, 300), (1, 296), (2, None), (2, P(0x30000002)), (3, 7), (4, None),
        (4, P(0x40000008)), (5, 296), (5, 308), (6, None), (6, P(0x50000001)), (7, -1), (7, 1 << 25), (8, 0),
        (8, 1 << 23), (9, 0), (9, 1 << 19), (10, 3), (10, -1), (11, None), (11, P(0x70000002)), (12, 199),
        (11, X), (11, S), (11, W), (11, U)])
    assert lib.gptq_fp8_gemm(None, 0, None, 0, None, 0, None, 0, 200, 300, 0, None, 0, None) == 0


def test_gated_refusals(lib):
    #       x  ldx  xs lds Wg gs Wu us  ldw  m  n    d   act out y  ldy  ys ldys
    codes = (X, 304, S, 8, W, U, V, T, 304, 8, 200, 300, 0, 3, Y, 208, C, 8, None)
    values = codes[:13] + (1, Y, 200, None, 0, None)
    refused(lib.gptq_fp8_gated, codes, [
        (0, None), (0, UNALIGNED), (4, None), (5, None), (6, None), (7, None), (6, P(0x60000004)), (8, 312), (8, 288),
        (12, 2), (12, -1), (13, 4), (14, None), (14, P(0x70000008)), (15, 200), (15, 216), (16, None), (17, 7),
        (14, X), (14, V), (16, T), (16, Y), (16, P(0x20000002))])
    refused(lib.gptq_fp8_gated, values, [(13, 5), (14, P(0x70000001)), (15, 199), (16, C), (14, S)])
    assert lib.gptq_fp8_gated(None, 0, None, 0, None, None, None, None, 0, 0, 200, 300, 1, 3, None, 0, None, 0,
                              None) == 0


def test_token_logprobs_refusals(lib):
    #       logits dtype n vocab ld targets logp entropy top top_logp top_ids
    good = (X, 1, 4, 1000, 1024, T, Y, S, 5, U, V, None)
    refused(lib.gptq_token_logprobs, good, [
        (0, None), (0, P(0x10000001)), (1, 3), (2, -1), (2, 1 << 25), (3, 0), (3, 1 << 31), (4, 999), (4, 1 << 40),
        (5, None), (5, P(0x80000004)), (6, None), (6, P(0x70000002)), (7, P(0x30000001)), (8, -1), (8, 33), (9, None),
        (10, None), (9, P(0x50000001)), (10, P(0x60000002)), (8, 0), (6, X), (6, T), (7, Y), (9, X), (10, U)])
    refused(lib.gptq_token_logprobs, (X, 0, 4, 3, 3, T, Y, None, 3, U, V, None), [(8, 4)])
    assert lib.gptq_token_logprobs(None, 0, 0, 10, 10, None, None, None, 0, None, None, None) == 0


def test_reference_forms():
    """The tests' rounding is torch's on single-precision values, and goes to
    the nearer code where a double rounding would not."""
    rng = np.random.default_rng(0)
    q = np.clip(rng.normal(size=50000) * np.exp(3 * rng.normal(size=50000)), -448, 448).astype(np.float32)
    want = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(f8.e4m3_round(q.astype(np.float64)), want)
    assert np.array_equal(f8.TABLE[:127], torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double())
    tie = 1.0625                                   # between 1 (0x38) and 1.125 (0x39)
    assert list(f8.e4m3_round(np.array([tie, tie * (1 + 2.0 ** -40), tie * (1 - 2.0 ** -40)]))) == [0x38, 0x39, 0x38]
    x = np.array([[1.0, -448.0, 0.0, 2.0 ** -9] + [0.0] * 200])
    c, s = f8.quantize(x, 1)
    assert s.shape == (1, 2) and s[0, 0] == 1 and list(c[0, :4]) == [0x38, 0xFE, 0, 1]
    assert np.array_equal(f8.values(c, s, 1), x)
