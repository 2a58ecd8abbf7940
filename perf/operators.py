"""The operators of an FP8 scoring head, as cases that can be measured.

Four operators, each with its plain form in elementary torch operations (32-bit
arithmetic, rounded once at the end) and the call of this package that
computes it:

  quantize   per-token, per-128-block e4m3 quantization of activations
  gemm       product of e4m3 operands with an fp32 scale for each block of 128
  linear     the whole layer: quantize, then the product
  logprobs   log probabilities of given tokens, entropy and top alternatives

`own` selects which of the two `run` computes.
"""
import math

import torch

own = False

BLOCK = 128         # values of K (and, for weights, rows of N) that share a scale
E4M3_MAX = 448.0
DEVICE = "cuda"

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a small batch: latency counts
        {"name": "quantize 16x5120", "op": "quantize", "m": 16, "k": 5120, "x": "bf16", "pad": 0},
        # the input of a down projection for a full prefill batch
        {"name": "quantize 8192x17408", "op": "quantize", "m": 8192, "k": 17408, "x": "bf16", "pad": 0},
        # fp32 activations, an odd row count, a last block of 16, rows inside a wider buffer
        {"name": "quantize 1001x2576 f32", "op": "quantize", "m": 1001, "k": 2576, "x": "f32", "pad": 48},
        # decode, eight sequences: the weights are read once for few rows
        {"name": "gemm 8x5120x17408", "op": "gemm", "m": 8, "k": 5120, "n": 17408, "out": "bf16"},
        # prefill of 2048 tokens through an up projection of the smaller model class
        {"name": "gemm 2048x2560x9728", "op": "gemm", "m": 2048, "k": 2560, "n": 9728, "out": "bf16"},
        # ragged in every size, fp32 outputs
        {"name": "gemm 777x2576x5003 f32", "op": "gemm", "m": 777, "k": 2576, "n": 5003, "out": "f32"},
        # one token through a down projection: the single-sequence decode step
        {"name": "linear 1x17408x5120", "op": "linear", "m": 1, "k": 17408, "n": 5120, "x": "bf16", "out": "bf16"},
        # 64 sequences decoded together
        {"name": "linear 64x5120x17408", "op": "linear", "m": 64, "k": 5120, "n": 17408, "x": "bf16", "out": "bf16"},
        # a full prefill batch: the compute-bound end
        {"name": "linear 8192x5120x17408", "op": "linear", "m": 8192, "k": 5120, "n": 17408, "x": "bf16", "out": "bf16"},
        # one decoded token with the usual twenty alternatives
        {"name": "logprobs 1x131072 top 20", "op": "logprobs", "m": 1, "v": 131072, "x": "bf16", "given": 1,
         "top": 20, "masked": False, "pad": 0},
        # the letters of 64 multiple-choice questions under a mask, odd vocabulary, fp32 logits
        {"name": "logprobs 64x100003 f32", "op": "logprobs", "m": 64, "v": 100003, "x": "f32", "given": 4,
         "top": 5, "masked": True, "pad": 0},
        # every token of a prompt batch scored
        {"name": "logprobs 4096x131072", "op": "logprobs", "m": 4096, "v": 131072, "x": "bf16", "given": 1,
         "top": 5, "masked": False, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges: sizes over their logarithm, odd ones among them."""
    op = rng.choice(["quantize", "gemm", "gemm", "linear", "linear", "logprobs", "logprobs"])
    if op == "quantize":
        return {"op": op, "m": _log_int(rng, 1, 8192), "k": 16 * _log_int(rng, 16, 1088),
                "x": rng.choice(["bf16", "f32"]), "pad": 16 * rng.choice([0, 0, 1, 5])}
    if op in ("gemm", "linear"):
        most = 8192 * 5120 * 17408
        while True:
            c = {"op": op, "m": _log_int(rng, 1, 8192), "k": 16 * _log_int(rng, 16, 1088),
                 "n": _log_int(rng, 64, 17408), "out": rng.choice(["bf16", "bf16", "f32"])}
            if c["m"] * c["k"] * c["n"] <= most:
                break
        if op == "linear":
            c["x"] = rng.choice(["bf16", "bf16", "f32"])
        return c
    most = 4096 * 131072 * 2
    while True:
        c = {"op": op, "m": _log_int(rng, 1, 4096), "v": _log_int(rng, 1000, 262144),
             "x": rng.choice(["bf16", "f32"]), "given": rng.choice([0, 1, 1, 4, 7]),
             "top": rng.choice([0, 1, 5, 20, 32]), "masked": rng.random() < 0.3,
             "pad": rng.choice([0, 0, 61, 128])}
        if c["m"] * (c["v"] + c["pad"]) * (2 if c["x"] == "bf16" else 4) <= most:
            return c


# ----------------------------------------------------------------------- inputs
def _blocks(k):
    return -(-k // BLOCK)


def _activations(g, m, k, dtype, pad=0):
    """N(0, 1) with one channel in a hundred twenty times larger; rows inside a buffer `pad` wider."""
    x = torch.randn(m, k + pad, generator=g, device=DEVICE)
    loud = torch.rand(k + pad, generator=g, device=DEVICE) < 0.01
    x *= torch.where(loud, 20.0, 1.0)
    return x.to(DTYPES[dtype])[:, :k]


def _weights(g, n, k):
    """N(0, 0.02) as e4m3 with the scale absmax / 448 of each 128 x 128 block."""
    w = torch.randn(n, k, generator=g, device=DEVICE) * 0.02
    nb, kb = _blocks(n), _blocks(k)
    p = torch.zeros(nb * BLOCK, kb * BLOCK, device=DEVICE)
    p[:n, :k] = w
    p = p.view(nb, BLOCK, kb, BLOCK)
    scale = p.abs().amax(dim=(1, 3)) / E4M3_MAX
    q = (p / scale[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:n, :k]
    return q.to(torch.float8_e4m3fn).contiguous(), scale


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "quantize":
        s["inp"] = _activations(g, case["m"], case["k"], case["x"], case["pad"])
    elif op == "linear":
        s["inp"] = _activations(g, case["m"], case["k"], case["x"])
        s["w"], s["w_scale"] = _weights(g, case["n"], case["k"])
    elif op == "gemm":
        # operands as the quantizer leaves them: scales block-major, rows padded to four
        x = _activations(g, case["m"], case["k"], "bf16")
        q, scale = _plain_quantize(x)
        room = torch.empty(scale.shape[0], -(-case["m"] // 4) * 4, device=DEVICE)
        s["q"], s["scale"] = q, room[:, :case["m"]].copy_(scale)
        s["w"], s["w_scale"] = _weights(g, case["n"], case["k"])
    else:
        m, v = case["m"], case["v"]
        # logits of a language model: a broad bulk and a few tokens well above it
        x = torch.randn(m, v + case["pad"], generator=g, device=DEVICE) * 2.5
        peak = torch.randint(0, v, (m, 6), generator=g, device=DEVICE)
        x.scatter_add_(1, peak, torch.rand(m, 6, generator=g, device=DEVICE) * 14.0)
        x = x[:, :v]
        if case["masked"]:
            # a grammar allows a share of the vocabulary; every ninth row is left with nothing
            x[torch.rand(m, v, generator=g, device=DEVICE) < 0.7] = -math.inf
            x[8::9] = -math.inf
        s["logits"] = x.to(DTYPES[case["x"]])
        if case["pad"]:
            room = torch.zeros(m, v + case["pad"], device=DEVICE, dtype=DTYPES[case["x"]])
            s["logits"] = room[:, :v].copy_(s["logits"])
        ids = torch.randint(0, v, (m, case["given"]), generator=g, device=DEVICE)
        if case["given"]:
            ids[:, 0] = torch.where(torch.rand(m, generator=g, device=DEVICE) < 0.5, peak[:, 0], ids[:, 0])
        if case["given"] > 1:
            ids[::5, -1] = -1           # rows with fewer tokens asked for
        s["ids"] = ids
    return s


# ------------------------------------------------------------------ plain forms
def _plain_quantize(x):
    """s = absmax / 448 over each 128 values of a row, q = e4m3(x / s); a zero block gives s = 0, q = 0."""
    m, k = x.shape
    kb = _blocks(k)
    p = torch.zeros(m, kb * BLOCK, device=x.device)
    p[:, :k] = x.float()
    p = p.view(m, kb, BLOCK)
    s = p.abs().amax(dim=2) / E4M3_MAX
    y = torch.where(s[..., None] == 0, torch.zeros((), device=x.device), p / s[..., None])
    y = y.clamp(-E4M3_MAX, E4M3_MAX).view(m, kb * BLOCK)[:, :k]
    return y.to(torch.float8_e4m3fn), s.t().contiguous()


def _plain_gemm(q, scale, w, w_scale, dtype):
    """out = sum over blocks b of scale[b, m] * w_scale[n / 128, b] * (q . w over block b)."""
    n, k = w.shape
    a = q.float() * scale.t().repeat_interleave(BLOCK, 1)[:, :k]
    b = w.float() * w_scale.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return (a @ b.t()).to(dtype)


def _plain_logprobs(logits, ids, top):
    """log p[id] = x[id] - log sum exp x; entropy = -sum p log p; the `top` largest, ties to the lowest index.

    A row that is -inf everywhere: -inf, entropy 0, no alternatives (id -1). A row with NaN or +inf:
    NaN, no alternatives. An alternative of -inf has id -1; an id of -1 asks for nothing and gives 0."""
    x = logits.float()
    m, v = x.shape
    peak = x.amax(dim=1, keepdim=True)                    # NaN if any is
    empty, bad = peak == -math.inf, ~(peak < math.inf)
    shift = torch.where(empty | bad, torch.zeros_like(peak), peak)
    e = torch.exp(x - shift)
    total = e.sum(dim=1, keepdim=True)
    lse = shift + torch.log(total)                        # -inf for an empty row
    centred = torch.where(e > 0, x - shift, torch.zeros_like(x))
    entropy = torch.log(total) - (e * centred).sum(dim=1, keepdim=True) / total
    entropy = torch.where(empty, torch.zeros_like(entropy), entropy)
    nan = torch.full_like(peak, math.nan)
    entropy = torch.where(bad, nan, entropy)[:, 0]

    def minus_lse(y):
        return torch.where(bad, nan, torch.where(y == -math.inf, y, y - torch.where(empty, shift, lse)))

    given = minus_lse(torch.gather(x, 1, ids.clamp(0, v - 1)))
    given = torch.where(ids < 0, torch.zeros_like(given), given)
    given = torch.where(ids >= v, nan, given)
    if top:
        value, index = torch.sort(x, dim=1, descending=True, stable=True)
        value, index = value[:, :top], index[:, :top]
        index = torch.where((value == -math.inf) | bad, torch.full_like(index, -1), index)
        value = minus_lse(value)
    else:
        value, index = x.new_empty(m, 0), ids.new_empty(m, 0)
    return given, entropy, index, value


# ------------------------------------------------------------------------- pass
def run(state):
    op = state["op"]
    if own:
        import bit_quantized_gemm_gb300 as qg
        if op == "quantize":
            q, scale = qg.quantize_act_fp8(state["inp"])
            return {"q": q, "scale": scale}
        if op == "gemm":
            return qg.gemm_fp8(state["q"], state["scale"], state["w"], state["w_scale"],
                               out_dtype=DTYPES[state["out"]])
        if op == "linear":
            return qg.linear_fp8(state["inp"], state["w"], state["w_scale"], out_dtype=DTYPES[state["out"]])
        given, entropy, index, value = qg.token_logprobs(state["logits"], state["ids"], top=state["top"])
    elif op == "quantize":
        q, scale = _plain_quantize(state["inp"])
        return {"q": q, "scale": scale}
    elif op == "gemm":
        return _plain_gemm(state["q"], state["scale"], state["w"], state["w_scale"], DTYPES[state["out"]])
    elif op == "linear":
        q, scale = _plain_quantize(state["inp"])
        return _plain_gemm(q, scale, state["w"], state["w_scale"], DTYPES[state["out"]])
    else:
        given, entropy, index, value = _plain_logprobs(state["logits"], state["ids"], state["top"])
    return {"given": given, "entropy": entropy, "top_ids": index, "top": value}


def work(case):
    op, m = case["op"], case["m"]
    if op == "logprobs":
        size = 2 if case["x"] == "bf16" else 4
        return {"bytes": m * case["v"] * size + m * case["given"] * 12 + m * 4 + m * case["top"] * 12,
                "flops": 5 * m * case["v"]}
    k, kb = case["k"], _blocks(case["k"])
    size = 2 if case.get("x") == "bf16" else 4
    if op == "quantize":
        return {"bytes": m * k * (size + 1) + m * kb * 4, "flops": 3 * m * k}
    n = case["n"]
    a = m * k + m * kb * 4 if op == "gemm" else m * k * size
    out = m * n * (2 if case["out"] == "bf16" else 4)
    return {"bytes": a + n * k + _blocks(n) * kb * 4 + out, "flops": 2 * m * n * k}


# ------------------------------------------------------------ 64-bit definition
def _exact_quantize(x):
    m, k = x.shape
    d = x.double()
    q, scales = torch.zeros_like(d), []
    for b in range(0, k, BLOCK):
        part = d[:, b:b + BLOCK]
        s = part.abs().max(dim=1).values / E4M3_MAX
        y = part / torch.where(s > 0, s, torch.ones_like(s))[:, None]
        # nearest e4m3 value, ties to even: three mantissa bits down to exponent -6
        _, e = torch.frexp(y)
        step = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)
        q[:, b:b + BLOCK] = (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
        scales.append(s)
    return q, torch.stack(scales)


def _exact_gemm(q, scale, w, w_scale):
    q, w, scale, w_scale = q.double(), w.double(), scale.double(), w_scale.double()
    n, k = w.shape
    rows = torch.arange(n, device=w.device) // BLOCK
    cols = torch.arange(k, device=w.device) // BLOCK
    return torch.matmul(q * scale[cols].t(), (w * w_scale[rows][:, cols]).t())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        q, scale = _exact_quantize(s["inp"])
        return {"q": q, "scale": scale}
    if op == "gemm":
        return _exact_gemm(s["q"], s["scale"], s["w"], s["w_scale"])
    if op == "linear":
        # the quantized activations are part of the operator: in 32 bits, as defined
        q, scale = _plain_quantize(s["inp"])
        return _exact_gemm(q, scale, s["w"], s["w_scale"])
    x, ids, top = s["logits"].double(), s["ids"], case["top"]
    empty = torch.isinf(x).all(dim=1)
    lse = torch.logsumexp(x, dim=1)
    lp = x - torch.where(empty, torch.zeros_like(lse), lse)[:, None]
    p = torch.exp(lp)
    entropy = -torch.special.xlogy(p, p).sum(dim=1)
    entropy[empty] = 0.0
    rows = torch.arange(x.shape[0], device=x.device)[:, None]
    given = torch.where(ids >= 0, lp[rows, ids.clamp(min=0)], torch.zeros((), device=x.device, dtype=x.dtype))
    value = torch.topk(lp, top, dim=1).values if top else lp[:, :0]
    return {"given": given, "entropy": entropy, "top_ids": None, "top": value}
