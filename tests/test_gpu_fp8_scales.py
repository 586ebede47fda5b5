"""Products whose scales are far from one each but not their product: what
counts is xs[b][t] ws[r / 128][b], as the calls promise, whichever form runs.

All numbers here are powers of two or small multiples of them, so every step of
the sums is exact and the results are compared for equality, the activation's
apart (silu and gelu of such gates are the gate, to a rounding of the product)."""
import pytest
import torch

from post_weight_quantization_05_b200 import api, build_lib

pytestmark = pytest.mark.gpu

DEV = "cuda"
N, BLOCKS = 200, 3
D = 128 * BLOCKS
SUM = 2.0 ** 20                       # of a block: 128 x 2^6 x 2^7


@pytest.fixture(scope="module", autouse=True)
def _ready():
    build_lib.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    api.get_status(raise_on_error=False)
    yield
    code, _ = api.get_status(raise_on_error=False)
    assert code == 0


def codes(rows, value):
    return torch.full((rows, D), value, device=DEV).to(torch.float8_e4m3fn)


def scales(rows, value):
    return torch.full((BLOCKS, rows) if rows != N else (2, BLOCKS), value, device=DEV)


@pytest.mark.parametrize("m", [1, 20, 37, 300])
@pytest.mark.parametrize("ex,ew", [(110, -20), (-20, 110), (-126, 60), (60, -126), (120, -126)])
def test_product(m, ex, ew):
    y = torch.empty((m, N), device=DEV)
    api.fp8_gemm(codes(m, 64.0), scales(m, 2.0 ** ex), codes(N, 128.0), scales(N, 2.0 ** ew), y)
    assert (y == BLOCKS * SUM * 2.0 ** (ex + ew)).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m", [1, 20, 37, 300])
@pytest.mark.parametrize("large", ["gate", "up"])
def test_gated(m, act, large):
    """Token scales of 2^110: the gate's weights or the up projection's bring them
    back to 2^90, the other's to 2^-15."""
    eg, eu = (-20, -125) if large == "gate" else (-125, -20)
    y = torch.empty((m, N), device=DEV)
    api.fp8_gated(codes(m, 64.0), scales(m, 2.0 ** 110), codes(N, 128.0), scales(N, 2.0 ** eg), codes(N, 128.0),
                  scales(N, 2.0 ** eu), y, act=act)
    want = (BLOCKS * SUM * 2.0 ** (110 + eg)) * (BLOCKS * SUM * 2.0 ** (110 + eu))
    # three roundings at most of the activation and the product
    assert ((y.double() - want).abs() <= 4 * 2.0 ** -24 * want).all()
