"""Token scores on the GPU against 64 bits.

Tolerance: with d = x - M (one rounding), e^d comes from ex2 of d log2(e): one
rounding of the product (2^-24 |d| log2(e) ln 2 in the exponent, below 2^-23
|d|) and 2^-22 of the hardware function; a thread adds about vocab / 512 of
them, plus at most 40 additions and moves of the maximum in the joins (2^-23
each, a move being two roundings and one ex2).  So
  |ln S error| <= 2^-22 + 2^-23 E|d| + (vocab / 512 + 80) 2^-23
with E under p, and T = sum e^d d the same with E|d| and E d^2 in place of 1
and E|d|.  logp adds 2^-24 of |x - M| and of ln S, and one rounding of its own."""
import numpy as np
import pytest
import torch

from post_weight_quantization_05_b200 import api, build_lib

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


def scores(logits, targets, k=0):
    n = logits.shape[0]
    logp, ent = (torch.full((n,), 7.0, device="cuda") for _ in range(2))
    tl = torch.full((n, k), 7.0, device="cuda") if k else None
    ti = torch.full((n, k), -7, dtype=torch.int32, device="cuda") if k else None
    api.token_logprobs(logits, targets, logp, ent, tl, ti)
    return [None if t is None else t.cpu().numpy() for t in (logp, ent, tl, ti)]


def check(logits, targets, k=0):
    logp, ent, tl, ti = scores(logits, targets, k)
    x = logits.double().cpu().numpy()
    n, v = x.shape
    with np.errstate(all="ignore"):
        m = x.max(1, keepdims=True)
        d = x - m
        e = np.exp(d)
        s = e.sum(1)
        p = e / s[:, None]
        lp = d - np.log(s)[:, None]
        d0 = np.where(np.isfinite(d), d, 0)
    u = 2.0 ** -23
    adds = v / 512 + 80
    e1, e2 = (p * np.abs(d0)).sum(1), (p * d0 * d0).sum(1)
    ln_err = 2 * u + u * e1 + adds * u
    t = targets.cpu().numpy()
    rows = np.arange(n)
    want = np.where(t >= 0, lp[rows, np.maximum(t, 0)], 0.0)

    def near(got, ref, extra):
        fin = np.isfinite(ref)
        assert np.array_equal(got[~fin], ref[~fin].astype(np.float32))
        tol = extra + u * (np.abs(ref) + np.log(s).reshape(extra.shape[:1] + (1,) * (extra.ndim - 1)) + 1)
        assert (np.abs(got[fin] - ref[fin]) <= np.broadcast_to(tol, ref.shape)[fin]).all()
    near(logp, want, ln_err)
    h = -(p * np.where(np.isfinite(lp), lp, 0)).sum(1)
    near(ent, h, ln_err + e1 * (2 * u + adds * u) + u * e2 + e1 * ln_err)
    if k:
        order = np.argsort(-x, axis=1, kind="stable")[:, :k]
        assert np.array_equal(ti, order)
        near(tl, np.take_along_axis(lp, order, 1), ln_err[:, None])


def make(n, v, seed, dtype="fp32", ld=None, off=0):
    g = torch.Generator().manual_seed(seed)
    x = (2.5 * torch.randn((n, (ld or v) + off), generator=g)).to(DTYPES[dtype]).cuda()[:, off:off + v]
    return x, torch.randint(0, v, (n,), generator=g).cuda()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n,v,k", [(1, 1, 1), (3, 7, 7), (5, 31, 20), (2, 33, 32), (4, 511, 32), (3, 1000, 20),
                                   (2, 4095, 5), (5, 8192, 20), (3, 8193, 1), (2, 16400, 32), (1, 50257, 20),
                                   (3, 128000, 32), (700, 3001, 4)])
def test_rows(dtype, n, v, k):
    check(*make(n, v, v + n, dtype), k)


@pytest.mark.parametrize("dtype,ld,off", [("bf16", 50304, 0), ("bf16", 50257, 1), ("fp32", 50260, 3),
                                          ("fp16", 50263, 5)])
def test_pitched_and_misaligned(dtype, ld, off):
    check(*make(6, 50257, 1, dtype, ld, off), 5)


def test_no_top_and_no_entropy():
    x, t = make(9, 5000, 2)
    check(x, t, 0)
    a, b = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
    api.token_logprobs(x, t, a)
    api.token_logprobs(x, t, b, torch.empty(9, device="cuda"))
    assert torch.equal(a, b)


@pytest.mark.parametrize("v", [300, 9000, 40000])
def test_masks(v):
    """-inf and the type's lowest value in masked places; rows with one token
    left, with none left, and with none but the lowest value."""
    x, t = make(7, v, 3)
    x[0, ::2] = float("-inf")
    x[1, 5:] = float("-inf")
    x[2] = float("-inf")
    x[2, v - 1] = -3.0
    x[3, 3:] = torch.finfo(torch.float32).min
    x[4] = torch.finfo(torch.float32).min
    x[6, 1:] = 1e38
    t[1], t[2] = v - 1, v - 1
    check(x, t, 5)
    b = x[3:5].bfloat16()
    b[0, 3:] = torch.finfo(torch.bfloat16).min
    b[1] = torch.finfo(torch.bfloat16).min
    check(b, t[3:5], 5)


@pytest.mark.parametrize("v", [100, 9000, 128000])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_nothing_left(v, dtype):
    x, t = make(3, v, 4, dtype)
    x[1] = float("-inf")
    logp, ent, tl, ti = scores(x, t, 6)
    assert logp[1] == -np.inf and ent[1] == 0 and (tl[1] == -np.inf).all() and (ti[1] == np.arange(6)).all()
    assert np.isfinite(logp[[0, 2]]).all()
    check(x[[0, 2]], t[[0, 2]], 6)


@pytest.mark.parametrize("v", [600, 9000, 60000, 128000])
def test_ties_and_sorted_rows(v):
    """Equal values everywhere, both zeros, few distinct values, ascending and
    descending rows: equal values by increasing index."""
    x, t = make(7, v, 5)
    x[0] = 1.5
    x[1] = torch.where(torch.arange(v, device="cuda") % 3 == 0, -0.0, 0.0)
    x[2] = torch.randint(0, 4, (v,), generator=torch.Generator().manual_seed(1)).cuda().float()
    x[3] = torch.arange(v, device="cuda") * 1e-4
    x[4] = -torch.arange(v, device="cuda") * 1e-4
    x[5] = torch.arange(v, device="cuda") // 64 * 1e-2
    check(x, t, 32)
    check(x.bfloat16(), t, 20)


def test_nonfinite_rows():
    x, t = make(5, 9000, 6)
    x[1, 77] = float("nan")
    x[3, 8999] = float("inf")
    logp, ent, tl, ti = scores(x, t, 4)
    code, detail = api.get_status(raise_on_error=False)
    assert code == 4 and detail in (1, 3)
    for r in (1, 3):
        assert np.isnan(logp[r]) and np.isnan(ent[r]) and np.isnan(tl[r]).all() and (ti[r] == -1).all()
    check(x[[0, 2, 4]], t[[0, 2, 4]], 4)


def test_targets_not_scored_and_out_of_range():
    x, t = make(4, 1000, 7)
    t[1] = -100
    t[2] = 1000
    logp = scores(x, t)[0]
    code, detail = api.get_status(raise_on_error=False)
    assert (code, detail) == (1, 2)
    assert logp[1] == 0 and np.isnan(logp[2])
    check(x[[0, 3, 1]], t[[0, 3, 1]])


def test_same_bits_graph_and_stream():
    x, t = make(6, 60000, 8, "bf16")
    a, b, c = (torch.empty(6, device="cuda") for _ in range(3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    api.token_logprobs(x, t, a, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.token_logprobs(x, t, b)
    graph.replay()
    api.token_logprobs(x, t, c)
    assert torch.equal(a, b) and torch.equal(b, c)


def test_offsets_past_32_bits():
    """A pitched row whose first element lies behind 2^32 elements."""
    v, rows = 1000, 5
    ld = 1 << 30
    buf = torch.empty(((rows - 1) * ld + v,), dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((rows, v), (ld, 1))
    src, t = make(rows, v, 9, "bf16")
    x.copy_(src)
    check(x, t, 3)


def test_refusals():
    x, t = make(4, 100, 1)
    o = torch.empty(4, device="cuda")
    ids = torch.empty((4, 40), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        api.token_logprobs(x, t.int(), o)
    with pytest.raises(ValueError):
        api.token_logprobs(x, t, o[:3])
    with pytest.raises(ValueError):
        api.token_logprobs(x, t, o, None, torch.empty((4, 2), device="cuda"))
    with pytest.raises(ValueError):
        api.token_logprobs(x.t(), t, o)
    with pytest.raises(api.GPTQError):
        api.token_logprobs(x, t, o, None, torch.empty((4, 40), device="cuda"), ids)       # more than 32
    with pytest.raises(api.GPTQError):
        api.token_logprobs(x[:, :3], t, o, None, torch.empty((4, 5), device="cuda"), ids[:, :5].contiguous())
    api.token_logprobs(x[:0], t[:0], o[:0])
