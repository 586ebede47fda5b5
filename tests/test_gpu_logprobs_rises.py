"""Token scores of rows whose logits rise behind their first values, so that the
sums move to larger maxima on the way, against 64 bits.

Tolerance, from the sums in base 2 (u = 2^-24, the rounding of fp32).  A value
enters as e = 2^z with z = x log2(e) - k rounded once, and no value that counts
has |z| above |d| log2(e) + 17, d = x - M: k is moved to a piece's maximum where
that lies higher, before the piece is added if it lies more than 16 higher, and
k is rounded up to an integer.  Relative error of a value's e:
    2^-22 (ex2) + u (11.8 + |d|) (z's rounding, 17 ln 2 = 11.8) + u |d| / 2 (log2 e's)
and the joins' two factors add 2^-22 + 2 u |d| each, so
    eps(d) = 3 2^-22 + u (14 + 6 |d|)   (generous).
Additions: 32 in a piece per lane of a pair, one per piece, at most 15 in the
joins: A.  Those of S = sum e are relative to S, those of T = sum e d to
E|d| + 24 (z reaches 17 and a move adds up to 17, in units of ln 2).  Then
    ln S:  E[eps] + A u + 2 u |ln S| (logf, to a unit in the last place)
    T / S: E[|d| eps] + E|d| (E[eps] + A u) + A u (E|d| + 24) + 4 u (E|d| + 12)
and their difference and logp round once more each."""
import pytest
import torch

from post_weight_quantization_05_b200 import api, build_lib

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
VOCAB = 50257


@pytest.fixture(scope="module", autouse=True)
def _ready():
    build_lib.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    api.get_status(raise_on_error=False)
    yield
    code, _ = api.get_status(raise_on_error=False)
    assert code == 0


def check(x, targets):
    n, v = x.shape
    logp, ent = torch.empty((n,), device="cuda"), torch.empty((n,), device="cuda")
    tl, ti = torch.empty((n, 3), device="cuda"), torch.empty((n, 3), dtype=torch.int32, device="cuda")
    api.token_logprobs(x, targets, logp, ent, tl, ti)
    w = x.double()
    d = w - w.amax(1, keepdim=True)
    lns = torch.logsumexp(d, 1)
    p = torch.exp(d - lns[:, None])
    a = d.abs()
    e1, e2 = (p * a).sum(1), (p * a * a).sum(1)
    adds = (32 + -(-v * x.element_size() // 16384) + 15) * U
    eps = 3 * 2.0 ** -22 + 14 * U + 6 * U * e1
    ln_tol = eps + adds + 2 * U * lns
    t_tol = (3 * 2.0 ** -22 + 14 * U) * e1 + 6 * U * e2 + e1 * (eps + adds) + adds * (e1 + 24) + 4 * U * (e1 + 12)
    h = lns + e1
    assert ((ent.double() - h).abs() <= ln_tol + t_tol + 2 * U * (h + lns)).all()
    assert (ent >= 0).all()
    want = d.gather(1, targets[:, None])[:, 0] - lns
    assert ((logp.double() - want).abs() <= ln_tol + 2 * U * (want.abs() + lns)).all()
    assert (logp <= 0).all() and (tl <= 0).all()
    order = torch.sort(w, dim=1, descending=True, stable=True)[1][:, :3]
    assert torch.equal(ti.long(), order)
    want = d.gather(1, order) - lns[:, None]
    assert ((tl.double() - want).abs() <= ln_tol[:, None] + 2 * U * (want.abs() + lns[:, None])).all()


RISES = (3.0, 5.5, 7.9, 10.0, 20.0, 40.3, 45.0, 300.0)


def rows(kind, dtype, first, copies):
    """Every rise, `copies` times: the values from `first` on lie that much higher."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros((len(RISES) * copies, VOCAB), device="cuda")
    if kind == "random":
        x.normal_(generator=g).mul_(0.5)
    rise = torch.tensor(RISES, device="cuda").repeat(copies)[:, None]
    if kind == "peak":
        x[:, first + 77] += rise[:, 0]
    elif kind == "stairs":
        x += rise * (torch.arange(VOCAB, device="cuda") // first)
    else:
        x[:, first:] += rise
    x -= 30.0
    return x.to(dtype), torch.randint(0, VOCAB, (x.shape[0],), generator=g, device="cuda")


# a piece is 16 KB of a row: a row by itself has a block for each piece, one of
# many rows has one block for all
@pytest.mark.parametrize("kind", ["equal", "random", "peak", "stairs"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("pieces,copies", [(1, 60), (1, 1), (8, 1)])
def test_rises(kind, dtype, pieces, copies):
    first = 16384 // torch.finfo(dtype).bits * 8 * pieces
    if first + 77 >= VOCAB:
        first = VOCAB - 100
    x, t = rows(kind, dtype, first, copies)
    check(x, t)
    t.fill_(first + 77)
    check(x, t)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_every_height(dtype):
    """Equal logits that rise by anything between 0 and 45, many rows to a block."""
    first = 16384 // torch.finfo(dtype).bits * 8
    x = torch.full((600, VOCAB), -30.0, device="cuda")
    x[:, first:] += torch.linspace(0, 45, 600, device="cuda")[:, None]
    check(x.to(dtype), torch.full((600,), VOCAB - 1, device="cuda"))


@pytest.mark.parametrize("n", [2, 600])
def test_far_from_zero(n):
    """Rows about a value so large that fp32 holds few between it and the next."""
    for c in (1e7, 3.1e7, 3.3e8, 6.5e8, 1e12, 1e30):
        x = torch.full((n, VOCAB), c, device="cuda")
        x[1::2] = -c
        check(x, torch.zeros((n,), dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("vocab", [300, 1500, 5000, 50257])
def test_one_token_is_certain(vocab):
    """A row that a single token has to itself: probability one, so no more than
    0 for its logarithm and no less than 0 for the entropy."""
    x = torch.zeros((64, vocab), device="cuda")
    at = torch.arange(64, device="cuda") * (vocab // 64)
    x[torch.arange(64, device="cuda"), at] = torch.linspace(20, 60, 64, device="cuda")
    check(x, at)
    check(x - 31.7, at)
