"""Score tokens with an FP8 output head.

Hidden states go through the FP8 layer call (per-token, per-128-block e4m3
activations; e4m3 weights with a scale for each 128 x 128 block) to logits, and
token_logprobs reads off what a caller wants of them: the log probabilities of
the given tokens, the entropy of each distribution and its likeliest tokens.
Weights and hidden states are synthetic.

    python examples/score_tokens.py --tokens 512 --hidden 5120 --vocab 65536 --top 5
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import bit_quantized_gemm_gb300 as qg  # noqa: E402


def to_fp8_blocks(w):
    """fp32 [N, K] -> e4m3 [N, K] and the scale absmax / 448 of each 128 x 128 block."""
    n, k = w.shape
    nb, kb = -(-n // 128), -(-k // 128)
    p = torch.zeros(nb * 128, kb * 128, device=w.device)
    p[:n, :k] = w
    p = p.view(nb, 128, kb, 128)
    scale = p.abs().amax(dim=(1, 3)).clamp(min=1e-12) / 448.0
    q = (p / scale[:, None, :, None]).view(nb * 128, kb * 128)[:n, :k]
    return q.to(torch.float8_e4m3fn).contiguous(), scale


def score(hidden, head, head_scale, tokens, top=0, chunk=2048, allowed=None):
    """Log probabilities of tokens[i] after hidden[i] and the rows' entropies and `top` likeliest
    tokens, `chunk` rows of logits at a time. `allowed`: optional bool [V], the tokens that may follow."""
    parts = []
    for i in range(0, hidden.shape[0], chunk):
        logits = qg.linear_fp8(hidden[i:i + chunk], head, head_scale)
        if allowed is not None:
            logits.masked_fill_(~allowed, -math.inf)
        parts.append(qg.token_logprobs(logits, tokens[i:i + chunk], top=top))
    return [torch.cat(p) for p in zip(*parts)]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--vocab", type=int, default=65536)
    ap.add_argument("--top", type=int, default=5)
    ap.add_argument("--chunk", type=int, default=2048)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda")
    g.manual_seed(a.seed)
    head, head_scale = to_fp8_blocks(torch.randn(a.vocab, a.hidden, generator=g, device="cuda") * 0.05)
    hidden = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    tokens = torch.randint(0, a.vocab, (a.tokens,), generator=g, device="cuda")
    logprobs, entropy, ids, alternatives = score(hidden, head, head_scale, tokens, a.top, a.chunk)
    qg.check_device_error()
    print("tokens %d  mean log probability %.4f  perplexity %.4g  mean entropy %.4f nats" %
          (a.tokens, logprobs.mean().item(), math.exp(-logprobs.mean().item()), entropy.mean().item()))
    for i in range(min(3, a.tokens)):
        best = "  ".join("%d:%.3f" % (t, p) for t, p in zip(ids[i].tolist(), alternatives[i].tolist()))
        print("token %d: %d %.4f  likeliest %s" % (i, tokens[i].item(), logprobs[i].item(), best))
    return logprobs, entropy, ids, alternatives


if __name__ == "__main__":
    main()
