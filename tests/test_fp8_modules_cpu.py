"""What the 8-bit layers' modules settle on the host, without a GPU: the inputs
they refuse."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

from post_weight_quantization_05_b200 import fp8


def test_tangents_are_refused():
    """No tangent is computed: an input that carries one is refused, in no_grad too."""
    x = torch.randn(3, 16)
    with fwad.dual_level():
        dual = fwad.make_dual(x, torch.ones_like(x))
        assert fp8._rows(x).shape == (3, 16)
        with pytest.raises(RuntimeError):
            fp8._rows(dual)
        with torch.no_grad(), pytest.raises(RuntimeError):
            fp8._rows(dual)
    with pytest.raises(RuntimeError):
        torch.func.jvp(fp8._rows, (x,), (x,))
