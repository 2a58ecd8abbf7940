"""GPU test of the way from the norm to the experts: 8-bit rows and their scales gathered by expert, for numbers of
rows that are no multiple of four (rows of scales start on 16 bytes)."""
import pytest
import torch

import bit_quantized_gemm_gb300 as qg
from test_gpu_grouped import BF16, DEV, E4M3, bits, by_expert

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_quantized_gemm_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    yield
    qg.check_device_error()


@pytest.mark.parametrize("tokens,top", [(1, 1), (1, 3), (97, 2), (131, 3)])
def test_gathered_rows(tokens, top):
    k, f, experts = 640, 272, 9
    g = torch.Generator(device=DEV)
    g.manual_seed(tokens)
    x, residual = (torch.randn(tokens, k, generator=g, device=DEV).to(BF16) for _ in range(2))
    weight = 1 + 0.1 * torch.randn(k, generator=g, device=DEV)
    w = (torch.randn(experts, f, k, generator=g, device=DEV) * 100).clamp(-448, 448).to(E4M3)
    ws = torch.rand(experts, 3, 5, generator=g, device=DEV) * 4e-4 + 1e-5
    expert = torch.rand(tokens, experts, generator=g, device=DEV).topk(top, dim=1).indices.flatten()
    order = expert.argsort(stable=True)
    offsets = torch.cat([order.new_zeros(1), torch.bincount(expert, minlength=experts).cumsum(0)])
    token, rows = order // top, tokens * top
    q, s, _ = qg.rmsnorm_quantize_act_fp8(x, weight, 1e-6, residual=residual)
    q = q.view(torch.uint8)[token].view(E4M3)
    packed = s[:, token]
    s = torch.empty(s.shape[0], (rows + 3) // 4 * 4, device=DEV)[:, :rows].copy_(packed)
    got = qg.gemm_fp8_grouped(q, s, offsets, w, ws)
    assert torch.equal(bits(got), bits(by_expert(q, s, offsets, w, ws, torch.empty_like(got))))
    # every row is its token's product with its expert's weights
    one, one_s, _ = qg.rmsnorm_quantize_act_fp8(x[-1:], weight, 1e-6, residual=residual[-1:])
    for i in (token == tokens - 1).nonzero()[:, 0].tolist():
        e = int(expert[order[i]])
        assert torch.equal(bits(got[i:i + 1]), bits(qg.gemm_fp8(one, one_s, w[e], ws[e])))
    if rows % 4 and rows > 1:
        with pytest.raises(qg.QGError):     # (scales without that room are refused)
            qg.gemm_fp8_grouped(q, packed.contiguous(), offsets, w, ws)
