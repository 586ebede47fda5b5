"""What a program around the 8-bit layers and the token scores sets or leaves
behind: torch's default type, targets that are no tokens."""
import pytest
import torch
from torch import nn

from post_weight_quantization_05_b200 import api, build_lib, driver, fp8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _ready():
    build_lib.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    api.get_status(raise_on_error=False)
    yield
    code, _ = api.get_status(raise_on_error=False)
    assert code == 0


def linear(n, d, seed):
    m = nn.Linear(d, n, bias=False, device="cuda", dtype=torch.bfloat16)
    with torch.no_grad():
        m.weight.copy_(torch.randn((n, d), generator=torch.Generator().manual_seed(seed)) * d ** -0.5)
    return m


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float16, torch.float64])
def test_any_default_type(default):
    """Scales and scores are fp32 whatever torch's default type is."""
    lin, gate, up, down = linear(130, 256, 1), linear(384, 256, 2), linear(384, 256, 3), linear(256, 384, 4)
    x = torch.randn((2, 9, 256), generator=torch.Generator().manual_seed(5)).to("cuda", torch.bfloat16)
    t = torch.randint(0, 130, (2, 9), generator=torch.Generator().manual_seed(6)).cuda()

    def outputs():
        layer, mlp = fp8.Fp8Linear(lin), fp8.Fp8GatedMLP(gate, up, down)
        s = driver.token_scores([mlp], layer, [x], [t], top=2)
        assert s.logp.dtype == s.entropy.dtype == s.top_logp.dtype == torch.float32
        return layer(x), mlp(x), s.logp, s.entropy, s.top_logp, s.top_ids
    want = outputs()
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        got = outputs()
    finally:
        torch.set_default_dtype(before)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_targets_that_are_no_tokens():
    """A target beyond the vocabulary is the call's error, not the next one's:
    nothing is left in the status word."""
    head = linear(100, 64, 7)
    x = torch.randn((3, 8, 64), generator=torch.Generator().manual_seed(8)).to("cuda", torch.bfloat16)
    t = torch.randint(0, 100, (3, 8), generator=torch.Generator().manual_seed(9)).cuda()
    want = driver.token_scores([], head, [x], [t])
    for bad in (100, 1 << 40):
        wrong = t.clone()
        wrong[2, 5] = bad
        for rows in (4, 8192):
            with pytest.raises(ValueError):
                driver.token_scores([], head, [x, x], [t, wrong], max_rows=rows)
    assert api.get_status(raise_on_error=False)[0] == 0
    assert torch.equal(driver.token_scores([], head, [x], [t]).logp, want.logp)


def test_scores_in_a_graph():
    """Captured and replayed on other targets."""
    head = linear(100, 64, 7)
    x = torch.randn((8, 64), generator=torch.Generator().manual_seed(8)).to("cuda", torch.bfloat16)
    t = torch.arange(8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        driver.token_scores([], head, [x], [t])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = driver.token_scores([], head, [x], [t])
    t.add_(50)
    graph.replay()
    assert torch.equal(s.logp, driver.token_scores([], head, [x], [t]).logp)
