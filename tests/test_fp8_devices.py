"""Devices of the FP8 calls and of token_logprobs: every tensor of a call, and its
stream, on one device; the library is entered with that device current. On stand-ins
for tensors, streams and the library (no GPU)."""
import contextlib

import pytest
import torch

import bit_quantized_gemm_gb300 as qg
from bit_quantized_gemm_gb300 import _lib

E4M3, BF16, F32, I64 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int64


class Tensor:
    """What the binding asks of a tensor, without memory behind it."""

    def __init__(self, shape, dtype, device=0, stride=None, is_cuda=True):
        self.shape, self.dtype, self.index, self.is_cuda = torch.Size(shape), dtype, device, is_cuda
        self.step = tuple(stride) if stride else torch.empty(shape, device="meta").stride()
        self.device = torch.device("cuda", device) if is_cuda else torch.device("cpu")

    def get_device(self):
        return self.index if self.is_cuda else -1

    def dim(self):
        return len(self.shape)

    def stride(self):
        return self.step

    def is_contiguous(self):
        return self.step == torch.empty(self.shape, device="meta").stride()

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 0x10000


class Stream:
    cuda_stream = 77

    def __init__(self, device):
        self.device_index = device


class Library:
    """Records the device that is current at each call, and the call's stream."""

    def __init__(self):
        self.calls = []

    def qg_linear_fp8_workspace_bytes(self, M, K):
        return 1 << 20

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, _lib._current_device(), args[-1]))
            return _lib.QG_OK
        return fn


@pytest.fixture
def library(monkeypatch):
    lib, current = Library(), [0]

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    monkeypatch.setattr(_lib, "_lib", lib)
    monkeypatch.setattr(_lib, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(_lib, "_current_raw_stream", lambda index: 1000 + index)
    monkeypatch.setattr(_lib, "_empty", lambda shape, dtype, device, stream, ld=None: Tensor(
        shape, dtype, device.index, (ld, 1) if ld else None))
    return lib


M, K, N = 4, 256, 160


def arguments(device=0, **other):
    """Arguments of the four calls; `other`: devices of single ones."""
    def t(name, *a, **kw):
        return Tensor(*a, device=other.get(name, device), **kw)
    return dict(
        x=t("x", (M, K), BF16), q=t("q", (M, K), E4M3), scale=t("scale", (2, M), F32), w=t("w", (N, K), E4M3),
        w_scale=t("w_scale", (2, 2), F32), out=t("out", (M, N), F32), logits=t("logits", (M, N), F32),
        ids=t("ids", (M, 1), I64), workspace=t("workspace", (1 << 20,), torch.uint8))


def quantize(a, **kw):
    return qg.quantize_act_fp8(a["x"], out=(a["q"], a["scale"]), **kw)


def gemm(a, **kw):
    return qg.gemm_fp8(a["q"], a["scale"], a["w"], a["w_scale"], out=a["out"], **kw)


def linear(a, **kw):
    return qg.linear_fp8(a["x"], a["w"], a["w_scale"], out=a["out"], workspace=a["workspace"], **kw)


def logprobs(a, **kw):
    return qg.token_logprobs(a["logits"], a["ids"], top=2, **kw)


USES = [(quantize, ("x", "q", "scale")), (gemm, ("q", "scale", "w", "w_scale", "out")),
        (linear, ("x", "w", "w_scale", "out", "workspace")), (logprobs, ("logits", "ids"))]


@pytest.mark.parametrize("call", [u[0] for u in USES])
@pytest.mark.parametrize("device", [0, 1])
def test_the_tensors_device_is_current_in_the_call(library, call, device):
    call(arguments(device))
    call(arguments(device), stream=Stream(device))
    assert [c[1:] for c in library.calls] == [(device, 1000 + device), (device, 77)]
    assert _lib._current_device() == 0


@pytest.mark.parametrize("device", [0, 1])
def test_calls_that_allocate(library, device):
    a = arguments(device)
    qg.quantize_act_fp8(a["x"])
    qg.gemm_fp8(a["q"], a["scale"], a["w"], a["w_scale"])
    qg.linear_fp8(a["x"], a["w"], a["w_scale"])
    assert [c[1] for c in library.calls] == [device] * 3


@pytest.mark.parametrize("call,name", [(c, n) for c, names in USES for n in names])
def test_one_tensor_elsewhere_is_refused(library, call, name):
    with pytest.raises(ValueError):
        call(arguments(0, **{name: 1}))
    assert not library.calls


@pytest.mark.parametrize("call", [u[0] for u in USES])
def test_a_stream_of_another_device_is_refused(library, call):
    with pytest.raises(ValueError):
        call(arguments(0), stream=Stream(1))
    assert not library.calls


def test_a_workspace_of_host_memory_is_refused(library):
    a = arguments()
    a["workspace"] = Tensor((1 << 20,), torch.uint8, is_cuda=False)
    with pytest.raises(ValueError):
        linear(a)
    assert not library.calls


@pytest.mark.parametrize("shape,stride", [((1 << 20,), (0,)), ((1 << 10, 1 << 10), (1 << 11, 1)), ((1 << 20,), (2,))])
def test_a_workspace_that_is_not_one_piece_is_refused(library, shape, stride):
    # its element count says nothing of the memory from its first element on
    a = arguments()
    a["workspace"] = Tensor(shape, torch.uint8, stride=stride)
    with pytest.raises(ValueError):
        linear(a)
    assert not library.calls
