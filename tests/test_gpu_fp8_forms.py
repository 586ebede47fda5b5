"""Products whose forms meet more blocks of k than they keep scales for."""
import numpy as np
import pytest
import torch

from post_weight_quantization_05_b200 import api, build_lib
from test_gpu_fp8 import operands, reference, sum_tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    build_lib.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    api.get_status(raise_on_error=False)
    yield
    code, _ = api.get_status(raise_on_error=False)
    assert code == 0


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
