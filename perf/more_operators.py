"""The operators around the quantized projections of a serving model, as cases that can be measured.

Four operators, each with its plain form in elementary torch operations (32-bit
arithmetic, rounded once at the end) and the call of this package that
computes it:

  norm      root-mean-square norm, with the residual's addition, into 8-bit
            activations with their scales (e4m3 per token and 128 values, or
            int8 per token)
  gate      silu(gate) * up into e4m3 activations with their scales
  grouped   product of e4m3 operands with the weights of each row's expert, the
            rows sorted by expert, their numbers known on the device alone
  adapters  low-rank adapters of many requests added to a projection's output

`own` selects which of the two `run` computes.
"""
import math

import torch

own = False

BLOCK = 128         # values of K (and, for weights, rows of N) that share an e4m3 scale
E4M3_MAX = 448.0
DEVICE = "cuda"
EPS = 1e-6

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------ cases
def listed():
    return [
        # the token of a single sequence, before the projections of a layer: latency counts
        {"name": "norm 1x5120", "op": "norm", "form": "e4m3", "m": 1, "k": 5120, "x": "bf16", "weight": "bf16",
         "residual": True, "pad": 0},
        # a full prefill batch of the larger model class, with the residual's addition
        {"name": "norm 8192x5120", "op": "norm", "form": "e4m3", "m": 8192, "k": 5120, "x": "bf16", "weight": "bf16",
         "residual": True, "pad": 0},
        # the int8 layer's operand (its fp16 copy) from fp32 activations inside a wider buffer, an odd row count
        {"name": "norm int8 1001x2560 f32", "op": "norm", "form": "int8", "m": 1001, "k": 2560, "x": "f32",
         "weight": "f32", "residual": False, "pad": 48},
        # 64 sequences decoded together, between the two projections of an MLP
        {"name": "gate 64x9728", "op": "gate", "m": 64, "k": 9728, "x": "bf16", "pad": 0},
        # the same for a full prefill batch of the larger model class
        {"name": "gate 8192x17408", "op": "gate", "m": 8192, "k": 17408, "x": "bf16", "pad": 0},
        # one token at eight of 64 experts: gate and up of an expert an eighth as wide as the dense MLP
        {"name": "grouped 8 rows", "op": "grouped", "m": 8, "experts": 64, "k": 2560, "n": 2432, "out": "bf16"},
        # 64 sequences decoded together, eight experts each: nearly every expert is read for a few rows
        {"name": "grouped 512 rows", "op": "grouped", "m": 512, "experts": 64, "k": 2560, "n": 2432, "out": "bf16"},
        # down projections of a few experts, a last block of 64 values, an odd width, fp32 outputs
        {"name": "grouped 1777 rows f32", "op": "grouped", "m": 1777, "experts": 7, "k": 1216, "n": 2563, "out": "f32"},
        # 2048 prompt tokens, eight experts each: the compute-bound end
        {"name": "grouped 16384 rows", "op": "grouped", "m": 16384, "experts": 64, "k": 2560, "n": 2432, "out": "bf16"},
        # one token beside a down projection
        {"name": "adapters 1x17408x5120", "op": "adapters", "m": 1, "k": 17408, "n": 5120, "rank": 16, "adapters": 8,
         "x": "bf16", "out": "bf16", "runs": 1},
        # 64 requests decoded together, each with an adapter of its own or one of a few popular ones
        {"name": "adapters 64x5120x17408", "op": "adapters", "m": 64, "k": 5120, "n": 17408, "rank": 16, "adapters": 128,
         "x": "bf16", "out": "bf16", "runs": 64},
        # prompts of eleven requests in one batch, some without an adapter
        {"name": "adapters 4096x5120x17408", "op": "adapters", "m": 4096, "k": 5120, "n": 17408, "rank": 64,
         "adapters": 8, "x": "bf16", "out": "bf16", "runs": 11},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges: sizes over their logarithm, odd ones among them."""
    op = rng.choice(["norm", "gate", "grouped", "grouped", "adapters", "adapters"])
    while True:
        if op == "norm":
            form = rng.choice(["e4m3", "e4m3", "int8"])
            unit = 32 if form == "int8" else 16
            c = {"op": op, "form": form, "m": _log_int(rng, 1, 8192), "k": unit * _log_int(rng, 8, 17408 // unit),
                 "x": rng.choice(["bf16", "bf16", "f32"]), "weight": rng.choice(["bf16", "f32"]),
                 "residual": rng.random() < 0.7, "pad": 16 * rng.choice([0, 0, 1, 5])}
        elif op == "gate":
            c = {"op": op, "m": _log_int(rng, 1, 8192), "k": 16 * _log_int(rng, 16, 1088),
                 "x": rng.choice(["bf16", "bf16", "f32"]), "pad": 16 * rng.choice([0, 0, 1, 5])}
        elif op == "grouped":
            c = {"op": op, "m": _log_int(rng, 1, 16384), "experts": _log_int(rng, 1, 128),
                 "k": 16 * _log_int(rng, 16, 320), "n": _log_int(rng, 64, 5120), "out": rng.choice(["bf16", "bf16", "f32"])}
            if c["experts"] * c["k"] * c["n"] > 64 * 2560 * 2432:
                continue
        else:
            m = _log_int(rng, 1, 4096)
            c = {"op": op, "m": m, "k": 16 * _log_int(rng, 16, 1088), "n": _log_int(rng, 64, 17408),
                 "rank": 8 * _log_int(rng, 1, 16), "adapters": _log_int(rng, 1, 128), "x": rng.choice(["bf16", "bf16", "f32"]),
                 "out": rng.choice(["bf16", "bf16", "f32"]), "runs": _log_int(rng, 1, min(m, 64))}
            if c["adapters"] * c["rank"] * (c["k"] + c["n"]) > 128 * 16 * 22528 * 2:
                continue
        w = work(c)
        if w["bytes"] <= 8192 * 17408 * 5.2 and w["flops"] <= 2 * 16384 * 2560 * 2432:
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


def _expert_weights(g, e, n, k):
    """N(0, 0.02) as e4m3 with the scale absmax / 448 of each 128 x 128 block of each expert."""
    nb, kb = _blocks(n), _blocks(k)
    q = torch.empty(e, n, k, dtype=torch.float8_e4m3fn, device=DEVICE)
    scale = torch.empty(e, nb, kb, device=DEVICE)
    for i in range(e):
        p = torch.zeros(nb * BLOCK, kb * BLOCK, device=DEVICE)
        p[:n, :k] = torch.randn(n, k, generator=g, device=DEVICE) * 0.02
        p = p.view(nb, BLOCK, kb, BLOCK)
        scale[i] = p.abs().amax(dim=(1, 3)) / E4M3_MAX
        q[i] = (p / scale[i][:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:n, :k].to(q.dtype)
    return q, scale


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    s = dict(case)
    if op == "norm":
        s["inp"] = _activations(g, m, k, case["x"], case["pad"])
        s["w"] = (1.0 + 0.2 * torch.randn(k, generator=g, device=DEVICE)).to(DTYPES[case["weight"]])
        # the stream of residuals is a few times as loud as one layer's output
        s["res"] = (4.0 * torch.randn(m, k, generator=g, device=DEVICE)).to(DTYPES[case["x"]]) if case["residual"] else None
    elif op == "gate":
        x = torch.randn(m, 2 * k + case["pad"], generator=g, device=DEVICE) * 2.0
        s["inp"] = x.to(DTYPES[case["x"]])[:, :2 * k]
    elif op == "grouped":
        # operands as the quantizer leaves them: scales block-major, rows padded to four
        q, scale = _plain_e4m3(_activations(g, m, k, "bf16").float())
        s["q"], s["scale"] = q, torch.empty(_blocks(k), -(-m // 4) * 4, device=DEVICE)[:, :m].copy_(scale)
        # experts are not equally popular; some may get no rows
        popular = torch.softmax(0.5 * torch.randn(case["experts"], generator=g, device=DEVICE), dim=0)
        expert = torch.multinomial(popular, m, replacement=True, generator=g)
        counts = torch.bincount(expert, minlength=case["experts"])
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        s["room"] = int(counts.max())   # for the plain form: rows of the largest expert
        s["w"], s["w_scale"] = _expert_weights(g, case["experts"], case["n"], k)
    else:
        n, r, count = case["n"], case["rank"], case["adapters"]
        s["inp"] = _activations(g, m, k, case["x"])
        s["base"] = torch.randn(m, n, generator=g, device=DEVICE).to(DTYPES[case["out"]])
        s["a"] = (torch.randn(count, r, k, generator=g, device=DEVICE) / math.sqrt(k)).to(torch.bfloat16)
        s["b"] = (torch.randn(count, n, r, generator=g, device=DEVICE) * 0.1).to(torch.bfloat16)
        s["scaling"] = 0.25 + torch.rand(count, generator=g, device=DEVICE)
        # runs of consecutive rows belong to a request; one request in eight has no adapter
        first = torch.rand(m, generator=g, device=DEVICE).argsort()[:case["runs"] - 1]
        run_of = torch.zeros(m, dtype=torch.int64, device=DEVICE).index_fill_(0, first, 1).cumsum(0)
        of_run = torch.randint(0, count, (case["runs"] + 1,), generator=g, device=DEVICE)
        of_run[torch.rand(case["runs"] + 1, generator=g, device=DEVICE) < 0.125] = -1
        s["ids"] = of_run[run_of] if m > 1 else of_run[:1].clamp(min=0)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_e4m3(y):
    """s = absmax / 448 over each 128 values of a row, q = e4m3(y / s); a zero block gives s = 0, q = 0."""
    m, k = y.shape
    kb = _blocks(k)
    p = torch.zeros(m, kb * BLOCK, device=y.device)
    p[:, :k] = y
    p = p.view(m, kb, BLOCK)
    s = p.abs().amax(dim=2) / E4M3_MAX
    v = torch.where(s[..., None] == 0, torch.zeros((), device=y.device), p / s[..., None])
    v = v.clamp(-E4M3_MAX, E4M3_MAX).view(m, kb * BLOCK)[:, :k]
    return v.to(torch.float8_e4m3fn), s.t().contiguous()


def _plain_int8(y):
    """s = absmax / 127 over a row, q = rint(y / s) as fp16; a zero row gives s = 0, q = 0."""
    s = y.abs().amax(dim=1) / 127.0
    v = torch.where(s[:, None] == 0, torch.zeros((), device=y.device), y / s[:, None])
    return v.round().clamp(-127, 127).to(torch.float16), s


def _plain_norm(x, residual, weight):
    """h = x + residual, as it is stored; y = h / sqrt(mean h^2 + eps) * weight."""
    h = x.float()
    total = None
    if residual is not None:
        total = (h + residual.float()).to(residual.dtype)
        h = total.float()
    y = h * (1.0 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)) * weight.float()
    return y, total


def _plain_gate(x):
    gate, up = x.float().chunk(2, dim=1)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_grouped(q, scale, offsets, room, w, w_scale, dtype):
    """out[m] = sum over blocks b of scale[b, m] * w_scale[e, n / 128, b] * (q[m] . w[e] over block b), e the expert
    whose rows offsets[e] <= m < offsets[e + 1] hold m."""
    m, k = q.shape
    e, n, _ = w.shape
    a = q.float() * scale.t().repeat_interleave(BLOCK, 1)[:, :k]
    row = torch.arange(m, device=q.device)
    expert = (row[:, None] >= offsets[None, 1:]).sum(dim=1)

    def values(w, w_scale):
        return w.float() * w_scale.repeat_interleave(BLOCK, 1)[:, :n].repeat_interleave(BLOCK, 2)[:, :, :k]

    if m <= e:      # fewer rows than experts: the weights of each row's expert
        mine = w.view(torch.uint8)[expert].view(w.dtype)
        return torch.bmm(a[:, None], values(mine, w_scale[expert]).transpose(1, 2))[:, 0].to(dtype)
    batch = torch.zeros(e, room, k, device=q.device)
    place = row - offsets[expert]
    batch[expert, place] = a
    return torch.bmm(batch, values(w, w_scale).transpose(1, 2))[expert, place].to(dtype)


def _plain_adapters(base, x, a, b, ids, scaling):
    """out = base + scaling[id] * (x . a[id]^T) . b[id]^T for rows whose id is not negative."""
    m, k = x.shape
    count, r, _ = a.shape
    n = b.shape[1]
    f = torch.where(ids >= 0, scaling[ids.clamp(min=0)], torch.zeros((), device=x.device))
    if m <= count:  # fewer rows than adapters: the adapter of each row
        h = torch.bmm(a[ids.clamp(min=0)].float(), x.float()[:, :, None])
        y = torch.bmm(b[ids.clamp(min=0)].float(), h)[:, :, 0]
    else:           # every adapter's products, each row's own kept
        h = (x.float() @ a.float().view(count * r, k).t()).view(m, count, r)
        h = torch.where((ids[:, None] == torch.arange(count, device=x.device))[..., None], h, torch.zeros((), device=x.device))
        y = h.view(m, count * r) @ b.float().transpose(1, 2).reshape(count * r, n)
    return (base.float() + f[:, None] * y).to(base.dtype)


# ------------------------------------------------------------------------- pass
def run(state):
    op = state["op"]
    if own:
        import bit_quantized_gemm_gb300 as qg
        if op == "norm" and state["form"] == "e4m3":
            q, scale, total = qg.rmsnorm_quantize_act_fp8(state["inp"], state["w"], EPS, residual=state["res"])
            return {"q": q, "scale": scale, "sum": total}
        if op == "norm":
            _, scale, _, q16, total = qg.rmsnorm_quantize_act(state["inp"], state["w"], EPS, residual=state["res"],
                                                              q16=True, int8=False)
            return {"q": q16, "scale": scale, "sum": total}
        if op == "gate":
            q, scale = qg.silu_mul_quantize_act_fp8(state["inp"])
            return {"q": q, "scale": scale}
        if op == "grouped":
            return qg.gemm_fp8_grouped(state["q"], state["scale"], state["offsets"], state["w"], state["w_scale"],
                                       out_dtype=DTYPES[state["out"]])
        return qg.add_lora(state["base"], state["inp"], state["a"], state["b"], state["ids"], state["scaling"])
    if op == "norm":
        y, total = _plain_norm(state["inp"], state["res"], state["w"])
        q, scale = _plain_e4m3(y) if state["form"] == "e4m3" else _plain_int8(y)
        return {"q": q, "scale": scale, "sum": total}
    if op == "gate":
        q, scale = _plain_e4m3(_plain_gate(state["inp"]))
        return {"q": q, "scale": scale}
    if op == "grouped":
        return _plain_grouped(state["q"], state["scale"], state["offsets"], state["room"], state["w"], state["w_scale"],
                              DTYPES[state["out"]])
    return _plain_adapters(state["base"], state["inp"], state["a"], state["b"], state["ids"], state["scaling"])


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    if op == "norm":
        size = 2 if case["x"] == "bf16" else 4
        kept = 1 if case["form"] == "e4m3" else 2       # e4m3, or the fp16 copy of int8
        scales = m * _blocks(k) * 4 if case["form"] == "e4m3" else m * 4
        streams = 3 if case["residual"] else 1          # x, residual, their sum
        return {"bytes": m * k * (streams * size + kept) + scales + k * (2 if case["weight"] == "bf16" else 4),
                "flops": 6 * m * k}
    if op == "gate":
        size = 2 if case["x"] == "bf16" else 4
        return {"bytes": m * k * (2 * size + 1) + m * _blocks(k) * 4, "flops": 6 * m * k}
    n = case["n"]
    out = m * n * (2 if case["out"] == "bf16" else 4)
    if op == "grouped":
        # experts that m independent choices reach, were they all equally popular
        read = case["experts"] * (1 - (1 - 1 / case["experts"]) ** m)
        return {"bytes": m * k + m * _blocks(k) * 4 + read * (n * k + _blocks(n) * _blocks(k) * 4) + out,
                "flops": 2 * m * n * k}
    count = case["adapters"]
    read = count * (1 - (1 - 1 / count) ** case["runs"])
    return {"bytes": m * k * (2 if case["x"] == "bf16" else 4) + read * case["rank"] * (k + n) * 2 + 2 * out + m * 8,
            "flops": 2 * m * case["rank"] * (k + n)}


# ------------------------------------------------------------ 64-bit definition
def _exact_e4m3(y):
    q, scales = torch.zeros_like(y), []
    for b in range(0, y.shape[1], BLOCK):
        part = y[:, b:b + BLOCK]
        s = part.abs().max(dim=1).values / E4M3_MAX
        v = part / torch.where(s > 0, s, torch.ones_like(s))[:, None]
        # nearest e4m3 value, ties to even: three mantissa bits down to exponent -6
        _, e = torch.frexp(v)
        step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
        q[:, b:b + BLOCK] = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
        scales.append(s)
    return q, torch.stack(scales)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h, total = s["inp"].double(), None
        if s["res"] is not None:
            total = h + s["res"].double()
            h = total.to(s["res"].dtype).double()       # the sum is normalised as it is stored
        y = h / torch.sqrt(h.square().sum(dim=1) / case["k"] + EPS)[:, None] * s["w"].double()[None]
        if case["form"] == "e4m3":
            q, scale = _exact_e4m3(y)
        else:
            scale = y.abs().max(dim=1).values / 127
            q = torch.round(y / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None])
        return {"q": q, "scale": scale, "sum": total}
    if op == "gate":
        k = case["k"]
        gate, up = s["inp"][:, :k].double(), s["inp"][:, k:].double()
        q, scale = _exact_e4m3(gate * torch.sigmoid(gate) * up)
        return {"q": q, "scale": scale}
    if op == "grouped":
        cols = torch.arange(case["k"], device=DEVICE) // BLOCK
        rows = torch.arange(case["n"], device=DEVICE) // BLOCK
        out = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=DEVICE)
        edges = s["offsets"].tolist()
        for e in range(case["experts"]):
            lo, hi = edges[e], edges[e + 1]
            if hi > lo:
                a = s["q"][lo:hi].double() * s["scale"][cols, lo:hi].double().t()
                b = s["w"][e].double() * s["w_scale"][e].double()[rows][:, cols]
                out[lo:hi] = a @ b.t()
        return out
    out = s["base"].double()
    for i in s["ids"].unique().tolist():
        if i >= 0:
            mine = (s["ids"] == i).nonzero()[:, 0]
            h = s["inp"][mine].double() @ s["a"][i].double().t()
            out[mine] += float(s["scaling"][i]) * (h @ s["b"][i].double().t())
    return out
