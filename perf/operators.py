"""What the 8-bit floating-point layer and the token scores are measured on.

Four operators, as a program that serves or judges a quantized model calls them:

quantize  values to e4m3 codes with one fp32 scale per block of 128: per token
          and 128 input channels ("rows", the activations of each call), or
          per 128 x 128 block ("weight", once per layer)
product   y = x W^T from the codes of both sides
gated     h = act(x Wg^T) * (x Wu^T) from codes, as values or as the codes and
          scales that the next product takes
logprobs  the log probability of a given token for every position, the
          distribution's entropy and the k likeliest tokens

`run` computes them in plain torch operations (own = False) or through the
package's entry points (own = True); `exact` computes them in 64 bits.
"""
import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -90
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "fp8": 1}


def listed():
    return [
        # one decoding step's activations of a 4096-wide layer, eight sequences
        {"name": "rows decode", "op": "rows", "m": 8, "d_in": 4096, "pad": 0, "dtype": "bf16"},
        # a prompt chunk's hidden activations, in fp32 as an unfused forward leaves them, odd width
        {"name": "rows odd fp32", "op": "rows", "m": 1531, "d_in": 2309, "pad": 3, "dtype": "fp32"},
        # a long batch of prompts entering an 11008-wide down projection
        {"name": "rows prefill", "op": "rows", "m": 8192, "d_in": 11008, "pad": 0, "dtype": "bf16"},
        # the largest layer of the repository's workloads, quantized once when a model is loaded
        {"name": "weight large", "op": "weight", "d_out": 8192, "d_in": 28672, "dtype": "bf16"},
        # one token through the largest layer: the weight's bytes are the whole cost
        {"name": "product token", "op": "product", "m": 1, "d_out": 8192, "d_in": 28672, "out": "bf16"},
        # a ragged handful of sequences through an attention input projection, fp32 out
        {"name": "product small", "op": "product", "m": 37, "d_out": 2304, "d_in": 768, "out": "fp32"},
        # a chunk of prompts, ragged, through an up projection
        {"name": "product chunk", "op": "product", "m": 509, "d_out": 11008, "d_in": 4096, "out": "bf16"},
        # a long batch of prompts through the largest layer: bound by the tensor cores
        {"name": "product prefill", "op": "product", "m": 4096, "d_out": 8192, "d_in": 28672, "out": "bf16"},
        # one decoding step of four sequences through a gated feed-forward's first half
        {"name": "gated decode", "op": "gated", "m": 4, "d_ff": 11008, "d_in": 4096, "act": "silu", "out": "fp8"},
        # a batch of prompts through the same, straight to the next product's codes
        {"name": "gated prefill", "op": "gated", "m": 4096, "d_ff": 11008, "d_in": 4096, "act": "silu", "out": "fp8"},
        # one generated token's scores with twenty alternatives, part of the vocabulary masked
        {"name": "logprobs token", "op": "logprobs", "n": 1, "vocab": 128000, "top": 20, "masked": True,
         "dtype": "fp32"},
        # the perplexity of a batch of sequences over an odd vocabulary
        {"name": "logprobs batch", "op": "logprobs", "n": 8192, "vocab": 50257, "top": 5, "masked": False,
         "dtype": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["rows", "weight", "product", "product", "gated", "logprobs", "logprobs"])
    if op == "rows":
        d = _log_uniform(rng, 100, 28672)
        m = min(_log_uniform(rng, 1, 16384), 8192 * 11008 // d)
        return {"op": op, "m": m, "d_in": d, "pad": rng.choice([0, 0, 8, 1, 512]),
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "weight":
        return {"op": op, "d_out": _log_uniform(rng, 100, 8192), "d_in": _log_uniform(rng, 100, 28672),
                "dtype": rng.choice(["bf16", "fp32"])}
    if op == "logprobs":
        v = _log_uniform(rng, 1000, 200000)
        n = min(_log_uniform(rng, 1, 8192), 8192 * 50257 // v)
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        return {"op": op, "n": max(1, n * 2 // BYTES[dtype]), "vocab": v, "top": rng.choice([0, 1, 5, 20]),
                "masked": rng.random() < 0.3, "dtype": dtype}
    # widths in whole blocks more often than not, as layers have them; the rest carry padded rows
    d = _log_uniform(rng, 128, 28672)
    if rng.random() < 0.6:
        d = max(128, d // 128 * 128)
    n = _log_uniform(rng, 128, 11008)
    m = min(_log_uniform(rng, 1, 4096), max(1, 4096 * 8192 * 28672 // (2 * n * d)))
    if op == "product":
        return {"op": op, "m": m, "d_out": n, "d_in": d, "out": rng.choice(["bf16", "fp16", "fp32"])}
    return {"op": op, "m": m, "d_ff": n, "d_in": d, "act": rng.choice(["silu", "gelu"]),
            "out": rng.choice(["fp8", "bf16"])}


# ------------------------------------------------------------------- inputs
def _up(n, to):
    return -(-n // to) * to


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(m, d, g, dtype):
    """Tokens whose channels differ in scale, one channel in a hundred twenty
    times larger, as the inputs of a transformer's linear layers are."""
    x = torch.randn((m, d), generator=g, device="cuda")
    c = torch.exp(0.5 * torch.randn((d,), generator=g, device="cuda"))
    c *= 1 + 19 * (torch.rand((d,), generator=g, device="cuda") < 0.01)
    return (x * c).to(dtype)


def _padded(values, multiple):
    """`values` as the leading columns of rows whose pitch is a whole multiple."""
    m, d = values.shape
    buf = torch.zeros((m, _up(d, multiple)), dtype=values.dtype, device=values.device)
    buf[:, :d] = values
    return buf[:, :d]


def _scales(blocks):
    a = blocks.abs().amax(dim=(1, 3)).clamp(min=AMAX_FLOOR)
    return a / torch.full_like(a, E4M3_MAX)     # by a tensor: a division by a number multiplies by its reciprocal


def _input_codes(x, rows):
    """Codes and scales of x [m, d] as a program already holds them: blocks of
    1 x 128 (scales [blocks, m]) or of 128 x 128 (scales [row blocks, blocks])."""
    m, d = x.shape
    h = 1 if rows else BLOCK
    p = torch.zeros((_up(m, h), _up(d, BLOCK)), device=x.device)
    p[:m, :d] = x.float()
    p = p.view(-1, h, p.shape[1] // BLOCK, BLOCK)
    s = _scales(p)
    p /= s[:, None, :, None]
    c = p.clamp_(-E4M3_MAX, E4M3_MAX).view(_up(m, h), -1)[:m, :d].to(torch.float8_e4m3fn)
    return _padded(c, 16), s.t().contiguous() if rows else s


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    dev = {"device": "cuda"}
    if op == "rows":
        m, d, pad = case["m"], case["d_in"], case["pad"]
        s["x"] = _activations(m, d + pad, g, DTYPES[case["dtype"]])[:, :d]
        s["codes"] = torch.zeros((m, _up(d, 16)), dtype=torch.float8_e4m3fn, **dev)[:, :d]
        s["scales"] = torch.empty((_up(d, BLOCK) // BLOCK, m), **dev)
    elif op == "weight":
        n, d = case["d_out"], case["d_in"]
        s["W"] = (0.02 * torch.randn((n, d), generator=g, **dev)).to(DTYPES[case["dtype"]])
        s["codes"] = torch.zeros((n, _up(d, 16)), dtype=torch.float8_e4m3fn, **dev)[:, :d]
        s["scales"] = torch.empty((_up(n, BLOCK) // BLOCK, _up(d, BLOCK) // BLOCK), **dev)
    elif op in ("product", "gated"):
        m, d = case["m"], case["d_in"]
        n = case["d_out"] if op == "product" else case["d_ff"]
        s["x"], s["xs"] = _input_codes(_activations(m, d, g, torch.bfloat16), True)
        s["w"], s["ws"] = _input_codes(0.02 * torch.randn((n, d), generator=g, **dev), False)
        if op == "gated":
            s["u"], s["us"] = _input_codes(0.02 * torch.randn((n, d), generator=g, **dev), False)
        if case["out"] == "fp8":
            s["y"] = torch.zeros((m, _up(n, 16)), dtype=torch.float8_e4m3fn, **dev)[:, :n]
            s["ys"] = torch.empty((_up(n, BLOCK) // BLOCK, m), **dev)
        else:
            s["y"] = torch.empty((m, n), dtype=DTYPES[case["out"]], **dev)
            s["ys"] = None
    else:
        n, v, k = case["n"], case["vocab"], case["top"]
        # rows of a head padded to whole 128-byte lines; a few strong tokens in every row
        buf = torch.randn((n, _up(v, 64)), generator=g, **dev).mul_(2.5)
        buf += 3.0 * (torch.rand((n, 1), generator=g, **dev) < 0.5)
        hot = torch.randint(0, v, (n, 12), generator=g, **dev)
        buf.scatter_add_(1, hot, 9 * torch.rand((n, 12), generator=g, **dev))
        if case["masked"]:      # constrained decoding: seven tokens in ten may not come
            mask = torch.rand((1, buf.shape[1]), generator=g, **dev) < 0.7
            buf.masked_fill_(mask.scatter_(1, hot[:1], False), float("-inf"))
        s["logits"] = buf.to(DTYPES[case["dtype"]])[:, :v]
        s["targets"] = torch.where(torch.rand((n,), generator=g, **dev) < 0.7, hot[:, 0],
                                   torch.randint(0, v, (n,), generator=g, **dev))
        s["logp"], s["entropy"] = torch.empty((n,), **dev), torch.empty((n,), **dev)
        s["top_logp"] = torch.empty((n, k), **dev) if k else None
        s["top_ids"] = torch.empty((n, k), dtype=torch.int32, **dev) if k else None
    return s


# ------------------------------------------------------------------- plain
def _quantize(x, rows):
    """e4m3 codes of x / s, s the fp32 scale of each block. The quotient is
    taken in 64 bits so that a value beside the middle of two codes goes to
    the nearer one; the rounding is half to even on e4m3's spacing."""
    m, d = x.shape
    h = 1 if rows else BLOCK
    p = torch.zeros((_up(m, h), _up(d, BLOCK)), device=x.device)
    p[:m, :d] = x.float()
    p = p.view(-1, h, p.shape[1] // BLOCK, BLOCK)
    s = _scales(p)
    q = p.double() / s.double()[:, None, :, None]
    step = torch.exp2(torch.frexp(q)[1].clamp(min=-5).double() - 4)
    q = (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    c = q.view(_up(m, h), -1)[:m, :d].float().to(torch.float8_e4m3fn)
    return c, s.t().contiguous() if rows else s


def _widen(codes, scales, rows):
    """The values that codes and scales stand for."""
    m, d = codes.shape
    s = scales.t() if rows else scales.repeat_interleave(BLOCK, 0)[:m]
    return codes.float() * s.repeat_interleave(BLOCK, 1)[:, :d]


def _act(g, name):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.erf(g * 0.5 ** 0.5))


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("rows", "weight"):
        return _quantize(s["x"] if op == "rows" else s["W"], op == "rows")
    if op == "product":
        y = _widen(s["x"], s["xs"], True) @ _widen(s["w"], s["ws"], False).t()
        return y.to(DTYPES[case["out"]])
    if op == "gated":
        x = _widen(s["x"], s["xs"], True)
        h = _act(x @ _widen(s["w"], s["ws"], False).t(), case["act"]) * (x @ _widen(s["u"], s["us"], False).t())
        return _quantize(h, True) if case["out"] == "fp8" else h.to(DTYPES[case["out"]])
    x = s["logits"].float() + 0.0       # -0 and +0 are one value
    d = x - x.amax(1, keepdim=True)
    e = torch.exp(d)
    z = e.sum(1)
    out = {"logp": d.gather(1, s["targets"][:, None])[:, 0] - torch.log(z),
           "entropy": torch.log(z) - (e * d.clamp(min=-1e30)).sum(1) / z}
    if case["top"]:
        ids = torch.sort(x, dim=1, descending=True, stable=True)[1][:, :case["top"]]
        out["top_logp"] = d.gather(1, ids) - torch.log(z)[:, None]
        out["top_ids"] = ids.int()
    return out


# ------------------------------------------------------------------- the package's calls
def _run_own(s):
    from post_weight_quantization_05_b200 import api
    case = s["case"]
    op = case["op"]
    if op == "rows":
        api.fp8_quantize_rows(s["x"], s["codes"], s["scales"])
        return s["codes"], s["scales"]
    if op == "weight":
        api.fp8_quantize_weight(s["W"], s["codes"], s["scales"])
        return s["codes"], s["scales"]
    if op == "product":
        api.fp8_gemm(s["x"], s["xs"], s["w"], s["ws"], s["y"])
        return s["y"]
    if op == "gated":
        api.fp8_gated(s["x"], s["xs"], s["w"], s["ws"], s["u"], s["us"], s["y"], s["ys"], act=case["act"])
        return s["y"] if s["ys"] is None else (s["y"], s["ys"])
    api.token_logprobs(s["logits"], s["targets"], s["logp"], s["entropy"], s["top_logp"], s["top_ids"])
    out = {"logp": s["logp"], "entropy": s["entropy"]}
    if case["top"]:
        out["top_logp"], out["top_ids"] = s["top_logp"], s["top_ids"]
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- cost
def work(case):
    op = case["op"]
    blocks = lambda n: -(-n // BLOCK)  # noqa: E731
    if op == "rows":
        m, d = case["m"], case["d_in"]
        return {"bytes": m * d * (BYTES[case["dtype"]] + 1) + 4 * m * blocks(d), "flops": 2 * m * d}
    if op == "weight":
        n, d = case["d_out"], case["d_in"]
        return {"bytes": n * d * (BYTES[case["dtype"]] + 1) + 4 * blocks(n) * blocks(d), "flops": 2 * n * d}
    if op in ("product", "gated"):
        m, d = case["m"], case["d_in"]
        n, mats = (case["d_out"], 1) if op == "product" else (case["d_ff"], 2)
        scales = 4 * (m * blocks(d) + mats * blocks(n) * blocks(d) + (m * blocks(n) if case["out"] == "fp8" else 0))
        return {"bytes": m * d + mats * n * d + m * n * BYTES[case["out"]] + scales, "flops": 2 * mats * m * n * d}
    n, v, k = case["n"], case["vocab"], case["top"]
    return {"bytes": n * (v * BYTES[case["dtype"]] + 8 + 8 + 8 * k), "flops": 5 * n * v}


# ------------------------------------------------------------------- 64 bits
def _grid(q):
    """The nearest e4m3 value of q: eight steps to each power of two from 2^-6
    on, steps of 2^-9 below, ties to the even multiple, at most 448."""
    lower = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6)))
    lower = torch.where(torch.exp2(lower) > q.abs().clamp(min=2.0 ** -6), lower - 1, lower)
    unit = torch.exp2(lower - 3)
    n = q.abs() / unit
    whole = torch.floor(n)
    rest = n - whole
    up = (rest > 0.5) | ((rest == 0.5) & (torch.remainder(whole, 2) == 1))
    return torch.sign(q) * torch.clamp((whole + up.double()) * unit, max=448.0)


def _exact_codes(x, tall):
    """x in 64 bits -> code values and scales (held in 32 bits) over blocks `tall` rows high."""
    m, d = x.shape
    x = torch.nn.functional.pad(x, (0, -d % 128, 0, -m % tall))
    t = x.unfold(0, tall, tall).unfold(1, 128, 128)                     # [.., .., tall, 128]
    s = (t.abs().amax((2, 3)).clamp(min=2.0 ** -90) / 448.0).to(torch.float32).double()
    whole = s.repeat_interleave(tall, 0).repeat_interleave(128, 1)
    return _grid(x / whole)[:m, :d], s


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rows":
        c, scales = _exact_codes(s["x"].double(), 1)
        return c, scales.T.contiguous()
    if op == "weight":
        return _exact_codes(s["W"].double(), 128)
    if op in ("product", "gated"):
        x = s["x"].double() * s["xs"].double().repeat_interleave(128, 0)[:case["d_in"]].T
        y = torch.matmul(x, _exact_weight(s["w"], s["ws"]).T)
        if op == "product":
            return y
        y = y * torch.sigmoid(y) if case["act"] == "silu" else y * torch.special.ndtr(y)
        y = y * torch.matmul(x, _exact_weight(s["u"], s["us"]).T)
        if case["out"] != "fp8":
            return y
        c, scales = _exact_codes(y, 1)
        return c, scales.T.contiguous()
    x = s["logits"].double()
    lp = torch.log_softmax(x, 1)
    p = lp.exp()
    out = {"logp": lp[torch.arange(case["n"], device=lp.device), s["targets"]],
           "entropy": -torch.special.xlogy(p, p).sum(1)}
    if case["top"]:
        out["top_logp"] = torch.topk(lp, case["top"], dim=1).values
        out["top_ids"] = None
    return out


def _exact_weight(codes, scales):
    n, d = codes.shape
    return codes.double() * torch.kron(scales.double(), torch.ones((128, 128), dtype=torch.float64,
                                                                   device=codes.device))[:n, :d]
