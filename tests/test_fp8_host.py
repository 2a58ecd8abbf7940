"""Refusals of the FP8 calls and of token_logprobs: the C ABI validates on the
host before any launch; the binding checks the tensors it is given (no GPU)."""
import ctypes

import pytest
import torch

import bit_quantized_gemm_gb300 as qg
from bit_quantized_gemm_gb300 import _lib
from bit_quantized_gemm_gb300 import build as qbuild

P = ctypes.c_void_p
FAKE = 0x10000  # never dereferenced: every call below fails validation first
EINVAL, EALIGN = _lib.QG_EINVAL, _lib.QG_EALIGN


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return _lib.load()


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), EINVAL), (dict(q=0), EINVAL), (dict(s=0), EINVAL), (dict(dt=2), EINVAL),
    (dict(M=0), EINVAL), (dict(M=2**24 + 1), EINVAL), (dict(K=0), EINVAL), (dict(K=24, ldx=64), EINVAL),
    (dict(K=65536 + 16, ldx=70000), EINVAL), (dict(ldx=240), EINVAL), (dict(lds=3), EINVAL),
    (dict(lds=6), EALIGN), (dict(x=FAKE + 2), EALIGN), (dict(ldx=257), EALIGN), (dict(q=FAKE + 8), EALIGN),
    (dict(s=FAKE + 4), EALIGN), (dict(dt=1, ldx=258), EALIGN),
])
def test_quantize_refusals(L, kw, status):
    a = dict(x=FAKE, dt=0, M=4, K=256, ldx=256, q=FAKE, s=FAKE, lds=4)
    a.update(kw)
    assert L.qg_quantize_act_fp8(P(a["x"]), a["dt"], a["M"], a["K"], a["ldx"], P(a["q"]), P(a["s"]),
                                 a["lds"], None) == status
    assert L.qg_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), EINVAL), (dict(s=0), EINVAL), (dict(w=0), EINVAL), (dict(ws=0), EINVAL), (dict(out=0), EINVAL),
    (dict(M=0), EINVAL), (dict(N=0), EINVAL), (dict(N=2**24 + 1), EINVAL), (dict(K=200, ldw=256), EINVAL),
    (dict(ldw=240), EINVAL), (dict(ldo=15), EINVAL), (dict(dt=3), EINVAL), (dict(lds=2), EINVAL),
    (dict(lds=7), EALIGN), (dict(ldw=264), EALIGN), (dict(q=FAKE + 1), EALIGN), (dict(w=FAKE + 8), EALIGN),
    (dict(ws=FAKE + 2), EALIGN), (dict(out=FAKE + 8), EALIGN), (dict(s=FAKE + 8), EALIGN),
])
def test_gemm_refusals(L, kw, status):
    a = dict(q=FAKE, s=FAKE, lds=4, M=4, K=256, w=FAKE, ldw=256, ws=FAKE, N=16, out=FAKE, dt=0, ldo=16)
    a.update(kw)
    assert L.qg_gemm_fp8(P(a["q"]), P(a["s"]), a["lds"], a["M"], a["K"], P(a["w"]), a["ldw"], P(a["ws"]),
                         a["N"], P(a["out"]), a["dt"], a["ldo"], None) == status
    assert L.qg_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), EINVAL), (dict(w=0), EINVAL), (dict(ws=0), EINVAL), (dict(out=0), EINVAL), (dict(M=0), EINVAL),
    (dict(K=8), EINVAL), (dict(N=0), EINVAL), (dict(ldx=128), EINVAL), (dict(ldo=8), EINVAL),
    (dict(work=0), EINVAL), (dict(nbytes=-1), EINVAL), (dict(work=FAKE + 128), EALIGN),
    (dict(x=FAKE + 8), EALIGN), (dict(xdt=9), EINVAL), (dict(odt=9), EINVAL),
])
def test_linear_refusals(L, kw, status):
    a = dict(x=FAKE, xdt=0, M=4, K=256, ldx=256, w=FAKE, ldw=256, ws=FAKE, N=16, out=FAKE, odt=0, ldo=16,
             work=FAKE, nbytes=0)
    a.update(kw)
    need = L.qg_linear_fp8_workspace_bytes(4, 256)
    assert L.qg_linear_fp8(P(a["x"]), a["xdt"], a["M"], a["K"], a["ldx"], P(a["w"]), a["ldw"], P(a["ws"]),
                           a["N"], P(a["out"]), a["odt"], a["ldo"], P(a["work"]), need + a["nbytes"],
                           None) == status
    assert L.qg_last_error().decode()


def test_linear_workspace(L):
    # the scales of ceil(K/128) blocks for M rows up to a multiple of four, then M*K e4m3 values
    for M, K in [(1, 16), (3, 144), (64, 5120), (8192, 17408)]:
        scales = -(-K // 128) * (-(-M // 4) * 4) * 4
        up = lambda v: -(-v // 256) * 256  # noqa: E731
        assert L.qg_linear_fp8_workspace_bytes(M, K) == up(up(scales) + M * K)
    for M, K in [(0, 256), (4, 0), (4, 24), (4, 65552), (2**24 + 1, 16)]:
        assert L.qg_linear_fp8_workspace_bytes(M, K) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), EINVAL), (dict(dt=5), EINVAL), (dict(M=0), EINVAL), (dict(V=0), EINVAL),
    (dict(V=2**24 + 1, ldl=2**25), EINVAL), (dict(ldl=99), EINVAL), (dict(G=-1), EINVAL),
    (dict(G=2**16 + 1), EINVAL), (dict(ids=0), EINVAL), (dict(lp=0), EINVAL), (dict(top=33), EINVAL),
    (dict(top=-1), EINVAL), (dict(ti=0), EINVAL), (dict(tl=0), EINVAL),
    (dict(x=FAKE + 1), EALIGN), (dict(ids=FAKE + 4), EALIGN),
    (dict(ent=FAKE + 2), EALIGN), (dict(ti=FAKE + 4), EALIGN),
])
def test_logprobs_refusals(L, kw, status):
    a = dict(x=FAKE, dt=0, M=4, V=100, ldl=100, ids=FAKE, G=2, lp=FAKE, ent=FAKE, top=5, ti=FAKE, tl=FAKE)
    a.update(kw)
    assert L.qg_token_logprobs(P(a["x"]), a["dt"], a["M"], a["V"], a["ldl"], P(a["ids"]), a["G"], P(a["lp"]),
                               P(a["ent"]), a["top"], P(a["ti"]), P(a["tl"]), None) == status
    assert L.qg_last_error().decode()


def test_binding_refuses_tensors_it_cannot_use():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(16, 256).to(torch.float8_e4m3fn)
    ws = torch.zeros(1, 2)
    for call in [lambda: qg.quantize_act_fp8(x), lambda: qg.linear_fp8(x, w, ws),
                 lambda: qg.gemm_fp8(w, ws, w, ws),
                 lambda: qg.token_logprobs(x, torch.zeros(4, dtype=torch.int64))]:
        with pytest.raises(ValueError):     # host tensors
            call()
