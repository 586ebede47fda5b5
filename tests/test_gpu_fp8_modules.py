"""The 8-bit layers and the token scores as a model uses them: against the same
layers in 64 bits on the weights that their codes stand for."""
import numpy as np
import pytest
import torch
from torch import nn

import fp8_util as f8
from post_weight_quantization_05_b200 import api, build_lib, driver, fp8, gpt_block, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    build_lib.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    api.get_status(raise_on_error=False)
    yield
    code, _ = api.get_status(raise_on_error=False)
    assert code == 0


def linear(n, d, seed, bias=False, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    m = nn.Linear(d, n, bias=bias)
    with torch.no_grad():
        m.weight.copy_(torch.randn((n, d), generator=g) * d ** -0.5)
        if bias:
            m.bias.copy_(torch.randn((n,), generator=g))
    return m.to("cuda", dtype)


def quantized(x):
    """x [m, d] rounded through the activations' 8-bit form, in 64 bits."""
    c, s = f8.quantize(x.double().cpu().numpy(), 1)
    return f8.values(c, s, 1)


def weight_values(codes, scales):
    return f8.values(codes.contiguous().view(torch.uint8).cpu().numpy(), scales.cpu().numpy(), 128)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape,bias", [((5, 300), False), ((2, 40, 300), True), ((0, 300), True), ((300,), False)])
def test_linear(dtype, shape, bias):
    lin = linear(200, 300, 1, bias, dtype)
    layer = fp8.Fp8Linear(lin)
    x = torch.randn(shape, generator=torch.Generator().manual_seed(2)).to("cuda", dtype)
    y = layer(x)
    assert y.shape == (*shape[:-1], 200) and y.dtype == dtype
    if not x.numel():
        return
    xv, wv = quantized(x.reshape(-1, 300)), weight_values(layer.codes[:, :300], layer.codes_scales)
    ref, a = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    b = lin.bias.detach().double().cpu().numpy() if bias else 0.0
    # the product's rounding, then the sum's with the bias
    tol = (128 * 2.0 ** -23 + 12 * 2.0 ** -24) * a + torch.finfo(dtype).eps / 2 * (np.abs(ref) + np.abs(ref + b)) * 1.01
    assert (np.abs(y.double().cpu().numpy().reshape(-1, 200) - ref - b) <= tol + 2.0 ** -24).all()


def test_linear_takes_any_layout_and_refuses_gradients():
    layer = fp8.Fp8Linear(linear(130, 256, 3))
    x = torch.randn((64, 256), device="cuda").bfloat16()
    want = layer(x)
    assert torch.equal(layer(x.t().contiguous().t()), want)
    assert torch.equal(layer(torch.cat([x, x], 1)[:, :256]), want)
    state = {k: v.clone() for k, v in layer.state_dict().items()}
    other = fp8.Fp8Linear(linear(130, 256, 4))
    other.load_state_dict(state)
    assert torch.equal(other(x), want)
    other = other.half().to(torch.bfloat16)          # codes and scales are not the module's float type
    assert other.codes_scales.dtype == torch.float32 and torch.equal(other(x), want)
    with pytest.raises(RuntimeError):
        layer(x.float().requires_grad_())
    with torch.no_grad():
        layer(x.float().requires_grad_())


def test_linear_takes_rows_over_one_another():
    """Broadcast and overlapping rows are inputs like any other."""
    layer = fp8.Fp8Linear(linear(130, 256, 3))
    x = torch.randn((1, 256), device="cuda").bfloat16()
    assert torch.equal(layer(x.expand(9, 256)), layer(x.repeat(9, 1)))
    windows = torch.randn((1000,), device="cuda").bfloat16().unfold(0, 256, 8)
    assert torch.equal(layer(windows), layer(windows.contiguous()))


def test_quantize_linears_keeps_the_structure():
    """A linear held twice stays one, one given by itself is returned, and a
    subclass, whose weight its owner may read, stays."""
    class Own(nn.Linear):
        pass
    shared = linear(64, 64, 1)
    m = nn.Module()
    m.a, m.b, m.inner, m.own = shared, shared, nn.Sequential(shared, linear(64, 64, 2)), Own(64, 64)
    assert fp8.quantize_linears(m) is m
    assert isinstance(m.a, fp8.Fp8Linear) and m.a is m.b is m.inner[0] and m.inner[1] is not m.a
    assert type(m.own) is Own and isinstance(m.inner[1], fp8.Fp8Linear)
    assert isinstance(fp8.quantize_linears(linear(64, 64, 3)), fp8.Fp8Linear)


@pytest.mark.parametrize("m", [1, 20, 300])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_mlp(m, act):
    gate, up, down = linear(640, 384, 5), linear(640, 384, 6), linear(384, 640, 7)
    layer = fp8.Fp8GatedMLP(gate, up, down, act)
    x = torch.randn((m, 384), generator=torch.Generator().manual_seed(8)).cuda().bfloat16()
    y = layer(x).double().cpu().numpy()
    xv = quantized(x)
    g, u, d = (weight_values(getattr(layer, k), getattr(layer, k + "_scales")) for k in ("gate", "up", "down"))
    h = f8.act(xv @ g.T, act) * (xv @ u.T)
    ref = f8.values(*f8.quantize(h, 1), 1) @ d.T
    # codes of h next to the middle of two may go the other way: a step of at most
    # 2^-3 of the value for the few within 1e-5 of one (at most one in 2000 here)
    few = np.sqrt(1 / 2000) * 2.0 ** -3
    assert np.linalg.norm(y - ref) <= (few + 2.0 ** -8) * np.linalg.norm(ref)


def test_gated_mlp_refusals():
    with pytest.raises(ValueError):
        fp8.Fp8GatedMLP(linear(640, 384, 5), linear(512, 384, 6), linear(384, 640, 7))
    with pytest.raises(ValueError):
        fp8.Fp8GatedMLP(linear(640, 384, 5, bias=True), linear(640, 384, 6), linear(384, 640, 7))


def _model(d, heads, vocab, seed):
    blocks = gpt_block.gpt_stack(synth.gpt_stack_weights(2, d, base_seed=seed), heads, dtype=torch.float32)
    xs = [torch.from_numpy(x).cuda() for x in synth.gpt_stack_inputs(2, 2, 48, d, base_seed=seed)]
    head = linear(vocab, d, seed, dtype=torch.float32)
    g = torch.Generator().manual_seed(seed)
    targets = [torch.randint(0, vocab, x.shape[:2], generator=g).cuda() for x in xs]
    targets[1][0, :7] = -100
    return blocks, head, xs, targets


def test_token_scores_of_a_stack():
    """The scores are those of the logits that the model gives, whatever the
    chunks, and quantizing the stack changes them."""
    blocks, head, xs, targets = _model(256, 4, 1000, 11)
    s = driver.token_scores(blocks, head, xs, targets, top=3)
    with torch.no_grad():
        logits = torch.cat([head(blocks[1](blocks[0](x))).reshape(-1, 1000) for x in xs]).double()
    lp = torch.log_softmax(logits, 1)
    t = torch.cat([v.reshape(-1) for v in targets])
    want = torch.where(t >= 0, lp.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    # the scores' own rounding (a few units in the last place of values below 2^4)
    # and that of fp32 products of other shapes (256 terms of 1 / 16 each)
    assert (s.logp.double() - want).abs().max() <= 1e-4
    assert (s.entropy.double() + (lp.exp() * lp).sum(1)).abs().max() <= 1e-4
    assert torch.equal(s.scored, t >= 0) and int(s.scored.sum()) == t.numel() - 7
    top = lp.topk(3, 1)
    assert (s.top_logp.double() - top.values).abs().max() <= 1e-4
    assert abs(s.loss + float(want.sum() / (t >= 0).sum())) <= 1e-4
    assert abs(s.perplexity - np.exp(s.loss)) <= 1e-9 * s.perplexity
    small = driver.token_scores(blocks, head, xs, targets, max_rows=10)
    assert small.top_ids is None and (small.logp - s.logp).abs().max() <= 1e-4
    driver.BlockSequential(bits=3).quantize(blocks, xs)
    after = driver.token_scores(blocks, head, xs, targets)
    assert (after.logp - s.logp).abs().max() > 1e-3
    api.get_status()


def test_token_scores_of_a_head_that_transposes():
    blocks, head, xs, targets = _model(256, 4, 100, 14)
    want = driver.token_scores(blocks, head, xs, targets)
    got = driver.token_scores(blocks, lambda x: head(x).t().contiguous().t(), xs, targets)
    assert torch.equal(got.logp, want.logp) and torch.equal(got.entropy, want.entropy)


def test_token_scores_refusals():
    blocks, head, xs, targets = _model(256, 4, 100, 12)
    with pytest.raises(ValueError):
        driver.token_scores(blocks, head, xs, [t[:, 1:] for t in targets])
    with pytest.raises(ValueError):
        driver.token_scores(blocks, head, xs, targets[:1])
    with pytest.raises(ValueError):
        driver.token_scores(blocks, head, [], [])
    with pytest.raises(api.GPTQError):
        driver.token_scores(blocks, head, xs, targets, top=33)


def test_stack_in_8_bits():
    """A stack whose linears and head are replaced by their 8-bit forms stays
    near the float one: e4m3's rounding, 2^-4 of a value at most, enters at two
    operands of each product and goes through two residual blocks."""
    blocks, head, xs, targets = _model(256, 4, 1000, 13)
    with torch.no_grad():
        before = blocks[1](blocks[0](xs[0]))
    for b in blocks:
        fp8.quantize_linears(b)
        assert not driver.BlockSequential.linears(b) and isinstance(b.fc, fp8.Fp8Linear)
    with torch.no_grad():
        after = blocks[1](blocks[0](xs[0]))
    rel = float((after - before).norm() / before.norm())
    assert 0 < rel <= 2 * 2.0 ** -4
    q = driver.token_scores(blocks, fp8.Fp8Linear(head), xs, targets)
    assert torch.isfinite(q.logp).all() and torch.isfinite(q.entropy).all()
