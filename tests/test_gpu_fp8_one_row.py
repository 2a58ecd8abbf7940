"""GPU tests of single rows that lie in buffers of any pitch: there is no next row, so
the pitch takes no part in the call."""
import pytest
import torch

import bit_quantized_gemm_gb300 as qg

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
K, N = 400, 131


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_gemm_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    qg.check_device_error()


def in_buffer(t, pitch):
    """The one row of t as the first of a buffer of rows `pitch` apart."""
    room = torch.full((3, pitch), 9.0, device=DEV).to(t.dtype)
    room[:1, :t.shape[1]] = t
    return room, room[:1, :t.shape[1]]


@pytest.fixture(scope="module")
def data():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x = torch.randn(1, K, generator=g, device=DEV)
    w = (torch.randn(N, K, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    ws = torch.rand(2, 4, generator=g, device=DEV) * 1e-3
    return x, w, ws


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pitch", [K + 1, K + 3, K + 16])
def test_layer(data, dtype, pitch):
    x, w, ws = data
    x = x.to(dtype)
    q, s = qg.quantize_act_fp8(x)
    want = qg.linear_fp8(x, w, ws, out_dtype=dtype)
    row = in_buffer(x, pitch)[1]
    q2, s2 = qg.quantize_act_fp8(row)
    assert torch.equal(q2.float(), q.float()) and torch.equal(s2, s)
    assert torch.equal(qg.linear_fp8(row, w, ws, out_dtype=dtype), want)
    room, out = in_buffer(torch.zeros(1, N, device=DEV, dtype=dtype), N + pitch - K)
    qg.linear_fp8(row, w, ws, out=out)
    assert torch.equal(out, want)
    assert bool((room[0, N:] == 9).all()) and bool((room[1:] == 9).all())


@pytest.mark.parametrize("pitch", [K + 1, K + 16])
def test_gemm_operands(data, pitch):
    x, w, ws = data
    q, s = qg.quantize_act_fp8(x)
    want = qg.gemm_fp8(q, s, w, ws)
    assert torch.equal(qg.gemm_fp8(in_buffer(q.float(), pitch)[1].to(q.dtype).as_strided((1, K), (pitch, 1)), s, w, ws),
                       want)
    one = torch.empty(pitch, device=DEV).to(w.dtype).as_strided((1, K), (pitch, 1))
    one.copy_(w[:1])
    assert torch.equal(qg.gemm_fp8(q, s, one, ws[:1]), want[:, :1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_logprobs(dtype):
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    x = torch.randn(1, 5003, generator=g, device=DEV).to(dtype)
    ids = torch.tensor([[7, 5002]], device=DEV)
    want = qg.token_logprobs(x, ids, top=5)
    for pitch in (5004, 6007):
        assert all(torch.equal(a, b) for a, b in zip(qg.token_logprobs(in_buffer(x, pitch)[1], ids, top=5), want))
