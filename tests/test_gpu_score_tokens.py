"""The FP8 head and the log probabilities together, as examples/score_tokens.py
runs them: against the same steps in 64 bits from the layer's own logits, and
the layer's logits against its definition."""
import importlib.util
import math
import os

import pytest
import torch

import bit_quantized_gemm_gb300 as qg

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from bit_quantized_gemm_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("score_tokens", os.path.join(ROOT, "examples", "score_tokens.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens,chunk", [(1, 64), (50, 16), (300, 128)])
def test_scores(example, tokens, chunk):
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    head, scale = example.to_fp8_blocks(torch.randn(3001, 400, generator=g, device="cuda") * 0.05)
    hidden = torch.randn(tokens, 400, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.randint(0, 3001, (tokens,), generator=g, device="cuda")
    lp, entropy, top, alt = example.score(hidden, head, scale, ids, top=4, chunk=chunk)
    logits = qg.linear_fp8(hidden, head, scale).double()
    want = torch.log_softmax(logits, dim=1)
    rows = torch.arange(tokens, device="cuda")
    # 2e-5: the statistics' error bound of the log-probability tests
    assert float((lp.double() - want[rows, ids]).abs().max()) <= 2e-5
    assert float((entropy.double() + (want.exp() * want).sum(1)).abs().max()) <= 2e-5
    best = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :4]
    assert torch.equal(top, best)
    assert float((alt.double() - torch.gather(want, 1, best)).abs().max()) <= 2e-5


def test_a_mask_that_leaves_one_token_or_none(example):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    head, scale = example.to_fp8_blocks(torch.randn(1000, 256, generator=g, device="cuda"))
    hidden = torch.randn(7, 256, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.full((7,), 123, dtype=torch.int64, device="cuda")
    one = torch.zeros(1000, dtype=torch.bool, device="cuda")
    none = one.clone()
    one[123] = True
    lp, entropy, top, alt = example.score(hidden, head, scale, ids, top=2, allowed=one)
    assert bool((lp == 0).all()) and bool((entropy == 0).all())
    assert bool((top == torch.tensor([123, -1], device="cuda")).all())
    assert bool((alt == torch.tensor([0.0, -math.inf], device="cuda")).all())
    lp, entropy, top, alt = example.score(hidden, head, scale, ids, top=2, allowed=none)
    assert bool((lp == -math.inf).all()) and bool((entropy == 0).all()) and bool((top == -1).all())


def test_command(example, capsys):
    example.main(["--tokens", "9", "--hidden", "512", "--vocab", "2000", "--top", "3"])
    out = capsys.readouterr().out
    assert "perplexity" in out and "token 2:" in out
