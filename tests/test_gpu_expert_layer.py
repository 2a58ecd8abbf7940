"""GPU tests of the norm, the gate, the product grouped by expert and the adapters together: a layer
of experts and a projection with adapters, eagerly, on a stream of its own, captured and replayed."""
import pytest
import torch

import bit_quantized_gemm_gb300 as qg
from test_gpu_grouped import bits, by_expert
from test_gpu_lora import check as check_adapters
from test_gpu_norm_gate import check_e4m3, exact_norm, off_gate

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
T, K, F, E, TOP, N, R, L = 96, 640, 272, 9, 2, 384, 16, 5   # tokens, hidden, inner, experts, per token; projection, rank, adapters


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_gemm_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    qg.check_device_error()


def weights():
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    blocks = lambda v: -(-v // 128)  # noqa: E731

    def e4m3(*shape):
        return (torch.randn(*shape, generator=g, device=DEV) * 100).clamp(-448, 448).to(E4M3)

    def scales(*shape):
        return torch.rand(*shape, generator=g, device=DEV) * 4e-4 + 1e-5
    return dict(
        norm=1 + 0.1 * torch.randn(K, generator=g, device=DEV),
        up=e4m3(E, 2 * F, K), up_s=scales(E, blocks(2 * F), blocks(K)),
        down=e4m3(E, K, F), down_s=scales(E, blocks(K), blocks(F)),
        w=e4m3(N, K), w_s=scales(blocks(N), blocks(K)),
        a=(torch.randn(L, R, K, generator=g, device=DEV) / K ** 0.5).to(BF16),
        b=torch.randn(L, N, R, generator=g, device=DEV).to(BF16), scaling=0.5 + torch.rand(L, generator=g, device=DEV))


def inputs(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    expert = torch.rand(T, E, generator=g, device=DEV).topk(TOP, dim=1).indices.flatten()
    order = expert.argsort(stable=True)
    offsets = torch.cat([order.new_zeros(1), torch.bincount(expert, minlength=E).cumsum(0)])
    return dict(x=torch.randn(T, K, generator=g, device=DEV).to(BF16), res=(3 * torch.randn(T, K, generator=g, device=DEV)).to(BF16),
                rows=order // TOP, offsets=offsets, ids=torch.randint(-1, L, (T,), generator=g, device=DEV))


def layer(w, i, stream=None):
    """Norm, the experts' MLP on the sorted rows, and a projection with adapters."""
    q, s, total = qg.rmsnorm_quantize_act_fp8(i["x"], w["norm"], residual=i["res"], stream=stream)
    m = T * TOP
    mine = q.view(torch.uint8)[i["rows"]].view(E4M3)
    mine_s = torch.empty(s.shape[0], m, device=DEV).copy_(s[:, i["rows"]])
    up = qg.gemm_fp8_grouped(mine, mine_s, i["offsets"], w["up"], w["up_s"], stream=stream)
    q2, s2 = qg.silu_mul_quantize_act_fp8(up, stream=stream)
    down = qg.gemm_fp8_grouped(q2, s2, i["offsets"], w["down"], w["down_s"], out_dtype=F32, stream=stream)
    base = qg.linear_fp8(total, w["w"], w["w_s"], out_dtype=F32, stream=stream)
    y = qg.add_lora(base, total, w["a"], w["b"], i["ids"], w["scaling"], stream=stream)
    return dict(q=q, s=s, total=total, mine=mine, mine_s=mine_s, up=up, q2=q2, s2=s2, down=down, base=base, y=y)


def test_every_step_of_the_layer():
    w, i = weights(), inputs(1)
    o = layer(w, i)
    assert torch.equal(o["total"], (i["x"].float() + i["res"].float()).to(BF16))
    check_e4m3(o["q"], o["s"], exact_norm(o["total"], w["norm"], 1e-6), torch.tensor(2.0 ** -19, dtype=torch.float64, device=DEV))
    assert torch.equal(bits(o["up"]), bits(by_expert(o["mine"], o["mine_s"], i["offsets"], w["up"], w["up_s"], torch.empty_like(o["up"]))))
    gate, up = o["up"][:, :F].double(), o["up"][:, F:].double()
    check_e4m3(o["q2"], o["s2"], gate * torch.sigmoid(gate) * up, off_gate(gate))
    assert torch.equal(bits(o["down"]), bits(by_expert(o["q2"], o["s2"], i["offsets"], w["down"], w["down_s"], torch.empty_like(o["down"]))))
    check_adapters(o["y"], o["base"], o["total"], w["a"], w["b"], i["ids"], w["scaling"])


def same(a, b):
    return all(torch.equal(a[k].view(torch.uint8) if a[k].dtype == E4M3 else a[k],
                           b[k].view(torch.uint8) if b[k].dtype == E4M3 else b[k]) for k in a)


def test_on_another_stream():
    w, i = weights(), inputs(2)
    want = layer(w, i)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = layer(w, i)
        again = layer(w, i, stream=s)
    torch.cuda.synchronize()
    assert same(got, want) and same(again, want)


def test_captured_and_replayed_on_other_inputs():
    # the number of rows of each expert and the adapters change from replay to replay
    w, first = weights(), inputs(3)
    held = {k: v.clone() for k, v in first.items()}
    layer(w, held)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):      # two graphs of the same calls, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, layer(w, held)))
    for seed in (4, 5, 6):
        other = inputs(seed)
        if seed == 6:       # every row at one expert, no adapters
            other["offsets"] = torch.tensor([0] * E + [T * TOP], device=DEV)
            other["ids"].fill_(-1)
        for k in held:
            held[k].copy_(other[k])
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = layer(w, other)
        for _, got in graphs:
            assert same(got, want)


@pytest.mark.parametrize("rows", [40, 300])
def test_two_calls_at_once(rows):
    # on two streams, each with memory of its own; many times over
    w = weights()
    g = torch.Generator(device=DEV)
    g.manual_seed(rows)
    x = torch.randn(rows, K, generator=g, device=DEV).to(BF16)
    base = torch.randn(rows, N, generator=g, device=DEV).to(BF16)
    ids = [torch.randint(-1, L, (rows,), generator=g, device=DEV) for _ in range(2)]
    want = [qg.add_lora(base, x, w["a"], w["b"], i, w["scaling"]) for i in ids]
    q, s = qg.quantize_act_fp8(x)
    off = [torch.tensor([0] * 4 + [rows // 3] * 2 + [rows] * 4, device=DEV), torch.linspace(0, rows, E + 1, device=DEV).long()]
    want_g = [qg.gemm_fp8_grouped(q, s, o, w["up"], w["up_s"]) for o in off]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for j, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append((j, qg.add_lora(base, x, w["a"], w["b"], ids[j], w["scaling"]),
                            qg.gemm_fp8_grouped(q, s, off[j], w["up"], w["up_s"])))
    torch.cuda.synchronize()
    for j, y, up in got:
        assert torch.equal(y, want[j]) and torch.equal(bits(up), bits(want_g[j]))
