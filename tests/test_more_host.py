"""Refusals of the norm, the gate, the product grouped by expert and the adapters: the C ABI
validates on the host before any launch, the binding checks the tensors it is given; devices
and streams on stand-ins (no GPU)."""
import ctypes

import pytest
import torch

import bit_quantized_gemm_gb300 as qg
from bit_quantized_gemm_gb300 import _lib
from bit_quantized_gemm_gb300 import build as qbuild
from test_fp8_devices import BF16, E4M3, F32, I64, Stream, Tensor, library  # noqa: F401

P = ctypes.c_void_p
FAKE = 0x10000  # never dereferenced: every call below fails validation first
EINVAL, EALIGN = _lib.QG_EINVAL, _lib.QG_EALIGN


@pytest.fixture(scope="module")
def L():
    qbuild.build()
    return _lib.load()


NORM = [
    (dict(x=0), EINVAL), (dict(w=0), EINVAL), (dict(scale=0), EINVAL), (dict(res=0), EINVAL), (dict(sum=0), EINVAL),
    (dict(dt=2), EINVAL), (dict(wdt=2), EINVAL), (dict(M=0), EINVAL), (dict(M=2**24 + 1), EINVAL), (dict(K=0), EINVAL),
    (dict(K=40, ldx=64), EINVAL), (dict(K=65536 + 32, ldx=70000, ldr=70000, ldsum=70000), EINVAL),
    (dict(ldx=240), EINVAL), (dict(ldr=240), EINVAL), (dict(ldsum=240), EINVAL), (dict(eps=-1.0), EINVAL),
    (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL), (dict(x=FAKE + 8), EALIGN),
    (dict(res=FAKE + 4), EALIGN), (dict(sum=FAKE + 2), EALIGN), (dict(w=FAKE + 8), EALIGN), (dict(ldx=257), EALIGN),
    (dict(ldr=260), EALIGN), (dict(ldsum=258), EALIGN), (dict(q=FAKE + 8), EALIGN), (dict(scale=FAKE + 2), EALIGN),
]


@pytest.mark.parametrize("kw,status", NORM + [(dict(q=0), EINVAL), (dict(lds=3), EINVAL), (dict(lds=6), EALIGN)])
def test_norm_fp8_refusals(L, kw, status):
    a = dict(x=FAKE, res=FAKE, dt=0, M=4, K=256, ldx=256, ldr=256, w=FAKE, wdt=0, eps=1e-6, sum=FAKE, ldsum=256,
             q=FAKE, scale=FAKE, lds=4)
    a.update(kw)
    assert L.qg_rmsnorm_quantize_act_fp8(P(a["x"]), P(a["res"]), a["dt"], a["M"], a["K"], a["ldx"], a["ldr"], P(a["w"]),
                                         a["wdt"], a["eps"], P(a["sum"]), a["ldsum"], P(a["q"]), P(a["scale"]),
                                         a["lds"], None) == status
    assert L.qg_last_error().decode()


@pytest.mark.parametrize("kw,status", NORM + [
    (dict(q=0, q16=0), EINVAL), (dict(K=48, ldx=64, ldr=64, ldsum=64), EINVAL), (dict(q16=FAKE + 8), EALIGN),
    (dict(bs=FAKE + 2), EALIGN)])
def test_norm_int8_refusals(L, kw, status):
    a = dict(x=FAKE, res=FAKE, dt=0, M=4, K=256, ldx=256, ldr=256, w=FAKE, wdt=0, eps=1e-6, sum=FAKE, ldsum=256,
             q=FAKE, scale=FAKE, bs=FAKE, q16=FAKE)
    a.update(kw)
    assert L.qg_rmsnorm_quantize_act(P(a["x"]), P(a["res"]), a["dt"], a["M"], a["K"], a["ldx"], a["ldr"], P(a["w"]),
                                     a["wdt"], a["eps"], P(a["sum"]), a["ldsum"], P(a["q"]), P(a["scale"]), P(a["bs"]),
                                     P(a["q16"]), None) == status
    assert L.qg_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), EINVAL), (dict(q=0), EINVAL), (dict(s=0), EINVAL), (dict(dt=2), EINVAL), (dict(M=0), EINVAL),
    (dict(K=24, ldx=64), EINVAL), (dict(K=65552, ldx=140000), EINVAL), (dict(ldx=504), EINVAL), (dict(lds=3), EINVAL),
    (dict(lds=6), EALIGN), (dict(x=FAKE + 2), EALIGN), (dict(ldx=513), EALIGN), (dict(q=FAKE + 8), EALIGN),
    (dict(s=FAKE + 4), EALIGN),
])
def test_gate_refusals(L, kw, status):
    a = dict(x=FAKE, dt=0, M=4, K=256, ldx=512, q=FAKE, s=FAKE, lds=4)
    a.update(kw)
    assert L.qg_silu_mul_quantize_act_fp8(P(a["x"]), a["dt"], a["M"], a["K"], a["ldx"], P(a["q"]), P(a["s"]), a["lds"],
                                          None) == status
    assert L.qg_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), EINVAL), (dict(s=0), EINVAL), (dict(off=0), EINVAL), (dict(w=0), EINVAL), (dict(ws=0), EINVAL),
    (dict(out=0), EINVAL), (dict(M=0), EINVAL), (dict(E=0), EINVAL), (dict(E=1025), EINVAL), (dict(N=0), EINVAL),
    (dict(K=200), EINVAL), (dict(ldw=240), EINVAL), (dict(lde=4080), EINVAL), (dict(ldo=15), EINVAL), (dict(dt=3), EINVAL),
    (dict(lds=2), EINVAL), (dict(lds=7), EALIGN), (dict(ldw=264, lde=8000), EALIGN), (dict(lde=4104), EALIGN),
    (dict(q=FAKE + 1), EALIGN), (dict(off=FAKE + 4), EALIGN), (dict(w=FAKE + 8), EALIGN), (dict(ws=FAKE + 2), EALIGN),
    (dict(out=FAKE + 8), EALIGN), (dict(s=FAKE + 8), EALIGN),
])
def test_grouped_refusals(L, kw, status):
    a = dict(q=FAKE, s=FAKE, lds=4, M=4, K=256, off=FAKE, E=3, w=FAKE, ldw=256, lde=4096, ws=FAKE, N=16, out=FAKE, dt=0,
             ldo=16)
    a.update(kw)
    assert L.qg_gemm_fp8_grouped(P(a["q"]), P(a["s"]), a["lds"], a["M"], a["K"], P(a["off"]), a["E"], P(a["w"]), a["ldw"],
                                 a["lde"], P(a["ws"]), a["N"], P(a["out"]), a["dt"], a["ldo"], None) == status
    assert L.qg_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(base=0), EINVAL), (dict(x=0), EINVAL), (dict(a=0), EINVAL), (dict(b=0), EINVAL), (dict(ids=0), EINVAL),
    (dict(out=0), EINVAL), (dict(dt=2), EINVAL), (dict(xdt=2), EINVAL), (dict(M=0), EINVAL), (dict(M=2**20 + 1), EINVAL),
    (dict(K=8), EINVAL), (dict(N=0), EINVAL), (dict(count=0), EINVAL), (dict(count=2**20 + 1), EINVAL),
    (dict(rank=0), EINVAL), (dict(rank=12), EINVAL), (dict(rank=136), EINVAL), (dict(ldx=240), EINVAL),
    (dict(ldb=15), EINVAL), (dict(ldo=15), EINVAL), (dict(work=0), EINVAL), (dict(more=-1), EINVAL),
    (dict(work=FAKE + 128), EALIGN), (dict(x=FAKE + 8), EALIGN), (dict(base=FAKE + 1), EALIGN),
    (dict(out=FAKE + 1), EALIGN), (dict(a=FAKE + 8), EALIGN), (dict(b=FAKE + 8), EALIGN), (dict(ids=FAKE + 4), EALIGN),
    (dict(scaling=FAKE + 2), EALIGN),
])
def test_adapter_refusals(L, kw, status):
    a = dict(base=FAKE, dt=0, ldb=16, x=FAKE, xdt=0, M=4, K=256, ldx=256, a=FAKE, b=FAKE, count=2, rank=16, N=16, ids=FAKE,
             scaling=FAKE, out=FAKE, ldo=16, work=FAKE, more=0)
    a.update(kw)
    need = L.qg_add_lora_workspace_bytes(4, 256, 16)
    assert L.qg_add_lora(P(a["base"]), a["dt"], a["ldb"], P(a["x"]), a["xdt"], a["M"], a["K"], a["ldx"], P(a["a"]),
                         P(a["b"]), a["count"], a["rank"], a["N"], P(a["ids"]), P(a["scaling"]), P(a["out"]), a["ldo"],
                         P(a["work"]), need + a["more"], None) == status
    assert L.qg_last_error().decode()


def test_adapter_workspace(L):
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    # few rows: an fp32 sum for each part of K of 1024; more: eight, and three bf16 numbers
    for M, K, r in [(1, 16, 8), (64, 5120, 16), (128, 17408, 32), (7, 1040, 24), (32, 5120, 64), (16, 5120, 128)]:
        assert L.qg_add_lora_workspace_bytes(M, K, r) == up(-(-K // 1024) * M * r * 4)
    for M, K, r, padded in [(129, 16, 8, 16), (4096, 5120, 24, 32), (200, 5120, 72, 128), (33, 1024, 40, 64)]:
        assert L.qg_add_lora_workspace_bytes(M, K, r) == up(M * padded * 38)
    # a workspace of many rows is one of fewer
    for K in (16, 5120, 65536):
        for r in (8, 32, 40, 64, 72, 128):
            need = [L.qg_add_lora_workspace_bytes(M, K, r) for M in (1, 2, 15, 16, 17, 32, 33, 128, 129, 500, 2**20)]
            assert need == sorted(need) and need[0] > 0
    for M, K, r in [(0, 256, 16), (2**20 + 1, 256, 16), (4, 24, 16), (4, 256, 12), (4, 256, 136), (4, 0, 16)]:
        assert L.qg_add_lora_workspace_bytes(M, K, r) == 0


# ------------------------------------------------------------------ the binding
M, K, N, E, R = 4, 256, 160, 3, 16


def arguments(device=0, **other):
    """Arguments of the five calls; `other`: devices of single ones."""
    def t(name, *a, **kw):
        return Tensor(*a, device=other.get(name, device), **kw)
    return dict(
        x=t("x", (M, K), BF16), residual=t("residual", (M, K), BF16), weight=t("weight", (K,), F32),
        sum=t("sum", (M, K), BF16), q=t("q", (M, K), E4M3), scale=t("scale", (2, M), F32), q8=t("q8", (M, K), torch.int8),
        scale8=t("scale8", (M,), F32), bs=t("bs", (M, K // 32), torch.int32), q16=t("q16", (M, K), torch.float16),
        xx=t("xx", (M, 2 * K), BF16), offsets=t("offsets", (E + 1,), I64), w=t("w", (E, N, K), E4M3),
        w_scale=t("w_scale", (E, 2, 2), F32), out=t("out", (M, N), F32), base=t("base", (M, N), F32),
        a=t("a", (E, R, K), BF16), b=t("b", (E, N, R), BF16), ids=t("ids", (M,), I64), scaling=t("scaling", (E,), F32),
        workspace=t("workspace", (1 << 20,), torch.uint8))


def norm(a, **kw):
    return qg.rmsnorm_quantize_act_fp8(a["x"], a["weight"], residual=a["residual"], out=(a["q"], a["scale"], a["sum"]), **kw)


def norm8(a, **kw):
    return qg.rmsnorm_quantize_act(a["x"], a["weight"], residual=a["residual"],
                                   out=(a["q8"], a["scale8"], a["bs"], a["q16"], a["sum"]), **kw)


def gate(a, **kw):
    return qg.silu_mul_quantize_act_fp8(a["xx"], out=(a["q"], a["scale"]), **kw)


def grouped(a, **kw):
    return qg.gemm_fp8_grouped(a["q"], a["scale"], a["offsets"], a["w"], a["w_scale"], out=a["out"], **kw)


def adapters(a, **kw):
    return qg.add_lora(a["base"], a["x"], a["a"], a["b"], a["ids"], a["scaling"], out=a["out"], workspace=a["workspace"],
                       **kw)


USES = [(norm, ("x", "weight", "residual", "q", "scale", "sum")),
        (norm8, ("x", "weight", "residual", "q8", "scale8", "bs", "q16", "sum")), (gate, ("xx", "q", "scale")),
        (grouped, ("q", "scale", "offsets", "w", "w_scale", "out")),
        (adapters, ("base", "x", "a", "b", "ids", "scaling", "out", "workspace"))]
CALLS = [u[0] for u in USES]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("device", [0, 1])
def test_the_tensors_device_is_current_in_the_call(library, call, device):  # noqa: F811
    call(arguments(device))
    call(arguments(device), stream=Stream(device))
    assert [c[1:] for c in library.calls] == [(device, 1000 + device), (device, 77)]
    assert _lib._current_device() == 0


@pytest.mark.parametrize("call,name", [(c, n) for c, names in USES for n in names])
def test_one_tensor_elsewhere_is_refused(library, call, name):  # noqa: F811
    with pytest.raises(ValueError):
        call(arguments(0, **{name: 1}))
    assert not library.calls


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_device_is_refused(library, call):  # noqa: F811
    with pytest.raises(ValueError):
        call(arguments(0), stream=Stream(1))
    assert not library.calls


SHAPES = [
    (norm, "weight", (K + 1,), F32, None), (norm, "weight", (K,), torch.float16, None), (norm, "weight", (K,), F32, (2,)),
    (norm, "residual", (M, K), F32, None), (norm, "residual", (M, K - 16), BF16, None), (norm, "residual", (M, K), BF16, (1, M)),
    (norm, "sum", (M, K), F32, None), (norm, "sum", (M + 1, K), BF16, None), (norm, "q", (M, K), E4M3, (512, 1)),
    (norm, "scale", (M, 2), F32, None), (norm8, "q8", (M, K), torch.int8, (512, 1)), (norm8, "scale8", (M + 1,), F32, None),
    (norm8, "bs", (M, K), torch.int32, None), (norm8, "q16", (M, K), BF16, None), (gate, "xx", (M, 2 * K + 1), BF16, None),
    (gate, "q", (M, 2 * K), E4M3, None), (grouped, "offsets", (E,), I64, None), (grouped, "offsets", (E + 1,), torch.int32, None),
    (grouped, "offsets", (E + 1,), I64, (2,)), (grouped, "w", (N, K), E4M3, None), (grouped, "w", (E, N, K + 16), E4M3, None),
    (grouped, "w", (E, N, K), E4M3, (N * K, 1, N)), (grouped, "w_scale", (2, 2), F32, None), (grouped, "out", (M, N + 1), F32, None),
    (adapters, "x", (M + 1, K), BF16, None), (adapters, "a", (E, R, K), F32, None), (adapters, "a", (E, R, K - 16), BF16, None),
    (adapters, "b", (E, R, N), BF16, None), (adapters, "b", (E, N, R), BF16, (N * R * 2, R, 1)), (adapters, "ids", (M,), torch.int32, None),
    (adapters, "ids", (M, 1), I64, None), (adapters, "scaling", (E + 1,), F32, None), (adapters, "out", (M, N), BF16, None),
    (adapters, "workspace", (1 << 20,), torch.uint8, (0,)),
]


@pytest.mark.parametrize("call,name,shape,dtype,stride", SHAPES)
def test_shapes_types_and_strides_are_checked(library, call, name, shape, dtype, stride):  # noqa: F811
    a = arguments()
    a[name] = Tensor(shape, dtype, stride=stride)
    with pytest.raises(ValueError):
        call(a)
    assert not library.calls


def test_calls_that_allocate(library, monkeypatch):  # noqa: F811
    monkeypatch.setattr(_lib, "add_lora_workspace_bytes", lambda M, K, rank: 1 << 12)
    a = arguments(1)
    qg.rmsnorm_quantize_act_fp8(a["x"], a["weight"])
    qg.rmsnorm_quantize_act_fp8(a["x"], a["weight"], residual=a["residual"])
    qg.rmsnorm_quantize_act(a["x"], a["weight"], residual=a["residual"], block_sums=True, q16=True)
    qg.silu_mul_quantize_act_fp8(a["xx"])
    qg.gemm_fp8_grouped(a["q"], a["scale"], a["offsets"], a["w"], a["w_scale"])
    qg.add_lora(a["base"], a["x"], a["a"], a["b"], a["ids"])
    assert [c[1] for c in library.calls] == [1] * 6


def test_host_tensors_are_refused():
    x, e4m3 = torch.zeros(4, 256, dtype=BF16), torch.zeros(4, 256).to(E4M3)
    for call in [lambda: qg.rmsnorm_quantize_act_fp8(x, x[0]), lambda: qg.rmsnorm_quantize_act(x, x[0]),
                 lambda: qg.silu_mul_quantize_act_fp8(x),
                 lambda: qg.gemm_fp8_grouped(e4m3, torch.zeros(2, 4), torch.zeros(2, dtype=I64), e4m3[None],
                                             torch.zeros(1, 1, 2)),
                 lambda: qg.add_lora(x, x, x[None], x[None], torch.zeros(4, dtype=I64))]:
        with pytest.raises(ValueError):
            call()
