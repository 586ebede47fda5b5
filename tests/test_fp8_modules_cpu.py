"""What the 8-bit layers' modules settle on the host, without a GPU: the inputs
they refuse, how they move between devices and types, and which layers of a
model they replace."""
import pytest
import torch
import torch.autograd.forward_ad as fwad
from torch import nn

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


def held():
    """A module with a weight's buffers, as a layer has them."""
    m = fp8._Fp8Module()
    m.register_buffer("codes", torch.arange(32, dtype=torch.uint8).view(2, 16))
    m.register_buffer("codes_scales", torch.rand(1, 1))
    return m


def test_scales_keep_their_type():
    m = held()
    codes, scales = m.codes.clone(), m.codes_scales.clone()
    for change in (m.half, m.bfloat16, m.double, m.float, lambda: m.to("cpu", torch.bfloat16)):
        change()
        assert m.codes_scales.dtype == torch.float32 and torch.equal(m.codes_scales, scales)
        assert torch.equal(m.codes, codes)


def test_to_meta_and_back():
    """Buffers without memory get some, and a state dict fills them."""
    m = held()
    state = {k: v.clone() for k, v in m.state_dict().items()}
    m.to("meta")
    assert m.codes_scales.is_meta and m.codes.is_meta
    m.to_empty(device="cpu")
    m.load_state_dict(state)
    assert torch.equal(m.codes_scales, state["codes_scales"]) and m.codes_scales.dtype == torch.float32


def test_shared_memory():
    m = held()
    scales = m.codes_scales.clone()
    m.share_memory()
    assert m.codes_scales.is_shared() and m.codes.is_shared() and torch.equal(m.codes_scales, scales)


class Form(nn.Module):
    """Stands for Fp8Linear, which needs a GPU."""
    check = staticmethod(lambda linear: None)

    def __init__(self, linear):
        super().__init__()
        self.out_features, self.in_features = linear.weight.shape

    def forward(self, x):
        return x.new_zeros((*x.shape[:-1], self.out_features))


@pytest.mark.parametrize("nested", [False, True])
def test_encoder_layers_keep_their_linears(nested, monkeypatch):
    """torch's encoder layers read their linears' weights in inference: replaced,
    their forward would fail."""
    monkeypatch.setattr(fp8, "Fp8Linear", Form)
    layer = nn.TransformerEncoderLayer(32, 4, 64, batch_first=True)
    model = nn.Sequential(nn.TransformerEncoder(layer, 2) if nested else layer, nn.Linear(32, 8)).eval()
    x = torch.randn(2, 5, 32)
    with torch.no_grad():
        want = model[0](x)
        fp8.quantize_linears(model)
        assert isinstance(model[1], Form)
        assert torch.equal(model[0](x), want)
        assert model(x).shape == (2, 5, 8)


def test_excluded_linears_stay(monkeypatch):
    monkeypatch.setattr(fp8, "Fp8Linear", Form)
    shared = nn.Linear(8, 8)
    m = nn.Module()
    m.inner = nn.ModuleDict({"a": nn.Linear(8, 8), "b": nn.Linear(8, 8)})
    m.c, m.d = shared, shared
    seen = []
    fp8.quantize_linears(m, exclude=lambda name, linear: seen.append((name, linear)) or name in ("inner.a", "d"))
    assert type(m.inner.a) is nn.Linear and isinstance(m.inner.b, Form)
    assert isinstance(m.c, Form) and m.d is shared
    assert sorted(name for name, _ in seen) == ["c", "d", "inner.a", "inner.b"]
    lin = nn.Linear(4, 4)
    assert fp8.quantize_linears(lin, exclude=lambda name, _: name == "") is lin


def test_a_model_is_replaced_whole_or_not_at_all(monkeypatch):
    """A linear that has no 8-bit form is found before any other is replaced."""
    class Picky(Form):
        @staticmethod
        def check(linear):
            if linear.weight.dtype == torch.float64:
                raise ValueError("no")
    monkeypatch.setattr(fp8, "Fp8Linear", Picky)
    m = nn.Sequential(nn.Linear(8, 8), nn.Linear(8, 8).double())
    with pytest.raises(ValueError):
        fp8.quantize_linears(m)
    assert type(m[0]) is nn.Linear and type(m[1]) is nn.Linear
    fp8.quantize_linears(m, exclude=lambda name, linear: name == "1")
    assert isinstance(m[0], Picky) and type(m[1]) is nn.Linear


@pytest.mark.parametrize("linear", [nn.Linear(8, 8), nn.Linear(8, 8, dtype=torch.float64),
                                    nn.Linear(8, 8, device="meta")])
def test_linears_without_a_form(linear):
    """Weights off the GPU or of another type are refused."""
    with pytest.raises(ValueError):
        fp8.Fp8Linear.check(linear)
    with pytest.raises(ValueError):
        fp8.quantize_linears(linear)
    m = nn.ModuleList([linear])
    with pytest.raises(ValueError):
        fp8.quantize_linears(m)
    assert m[0] is linear
