"""The binding of the gated block and the checkpoint refuses tensors whose type, size or strides are not what
the kernels read (a C entry point sees bare pointers). On the CPU: tensors that say they are on device 0,
and no entry point behind them."""
import pytest
import torch

import gated_ref as R
from bit_gemm_wise_b200 import w4

M, H, K, G = 4, 16, 128, 128
BF16, F16, F32, U8, I8, I16, I32 = (torch.bfloat16, torch.float16, torch.float32, torch.uint8, torch.int8, torch.int16,
                                    torch.int32)


class Called(Exception):
    pass


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    def called(name, dev, stream, *args):
        raise Called(name)

    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(w4, "_call", called)


def arguments():
    t = lambda dtype, *shape: torch.zeros(*shape, dtype=dtype)
    w = lambda: [t(U8, H, K // 2), t(F16, H, K // G), t(I16, H, K // G)]
    return {"X": t(BF16, M, K), "Y": t(BF16, M, H), "dH": t(BF16, M, H), "dG": t(BF16, M, H), "dU": t(BF16, M, H),
            "dX": t(BF16, M, K), "dY": t(BF16, M, H), "X8": t(U8, M, K), "x_scale": t(U8, M, K // 32),
            "dW": t(BF16, H, K), "gate": w(), "up": w(), "weight": w(), "flags": 0}


def call(fn, a):
    ws = torch.zeros(1 << 16, dtype=U8)
    if fn == "gated":
        w4.w4a16_gated(a["X"], M, a["gate"], a["up"], H, K, G, "asym", "silu", a["Y"], ws)
    elif fn == "bwd":
        w4.w4a16_gated_bwd(a["dH"], M, a["gate"], a["up"], H, K, G, "asym", "silu", a["dG"], a["dU"], a["dX"], ws, X=a["X"])
    elif fn == "bwd8":
        w4.w4a16_gated_bwd(a["dH"], M, a["gate"], a["up"], H, K, G, "asym", "silu", a["dG"], a["dU"], a["dX"], ws,
                           X8=a["X8"], x_scale=a["x_scale"])
    elif fn == "dgrad":
        w4.w4a16_dgrad(a["dY"], M, a["weight"], H, K, G, "asym", a["dX"], ws)
    elif fn == "save":
        w4.fp8_ckpt_save(a["X"], M, K, a["X8"], a["x_scale"])
    elif fn == "load":
        w4.fp8_ckpt_load(a["X8"], a["x_scale"], M, K, a["X"])
    else:
        w4.fp8_ckpt_wgrad(a["dY"], a["X8"], a["x_scale"], M, H, K, a["dW"], a["flags"], ws)


WEIGHTS = {"gated": ["gate", "up"], "bwd": ["gate", "up"], "bwd8": ["gate", "up"], "dgrad": ["weight"]}
TENSORS = {"gated": ["X", "Y"], "bwd": ["dH", "X", "dG", "dU", "dX"], "bwd8": ["dH", "X8", "x_scale"], "dgrad": ["dY", "dX"],
           "save": ["X", "X8", "x_scale"], "load": ["X8", "x_scale", "X"], "wgrad": ["dY", "X8", "x_scale", "dW"]}


@pytest.mark.parametrize("fn,name", [(f, n) for f, names in TENSORS.items() for n in names])
def test_tensors(fn, name):
    """Types of the same size and larger ones: no check of bytes would notice."""
    for dtype in (I8, I32) if name in ("X8", "x_scale") else (F16, F32, I16, torch.float64):
        a = arguments()
        a[name] = a[name].to(dtype)
        with pytest.raises(ValueError, match=name + " is torch"):
            call(fn, a)


@pytest.mark.parametrize("fn,name", [(f, n) for f, names in WEIGHTS.items() for n in names])
@pytest.mark.parametrize("part,dtypes", [("codes", [I8, I32]), ("scales", [BF16, F32]), ("zeros", [F16, I32, U8])])
def test_weights(fn, name, part, dtypes):
    i = ["codes", "scales", "zeros"].index(part)
    for dtype in dtypes:
        a = arguments()
        a[name][i] = a[name][i].to(dtype)
        with pytest.raises(ValueError, match=f"{name} {part} is torch"):
            call(fn, a)


def test_dw_goes_by_the_flag():
    for flags, dtype in ((0, F32), (w4.W4_OUT_FP32, BF16)):
        a = arguments()
        a["flags"], a["dW"] = flags, torch.zeros(H, K, dtype=dtype)
        with pytest.raises(ValueError, match="dW is torch"):
            call("wgrad", a)


def test_types_that_hold_the_same_bits_are_taken():
    """Scales as w4_quantize's int16, E4M3 values and their scale bytes as such."""
    for fn in TENSORS:
        with pytest.raises(Called):
            call(fn, arguments())
    for name, dtype in (("X8", torch.float8_e4m3fn), ("x_scale", torch.float8_e8m0fnu)):
        for fn in ("save", "load", "wgrad", "bwd8"):
            a = arguments()
            a[name] = a[name].view(dtype)
            with pytest.raises(Called):
                call(fn, a)
    for dtype in (I16, torch.uint16):
        a = arguments()
        a["gate"][1] = a["gate"][1].view(dtype)
        with pytest.raises(Called):
            call("gated", a)
    a = arguments()
    a["flags"], a["dW"] = w4.W4_OUT_FP32, torch.zeros(H, K, dtype=F32)
    with pytest.raises(Called):
        call("wgrad", a)


PLACES = [(f, n, None) for f, names in TENSORS.items() for n in names] + \
         [(f, n, i) for f, names in WEIGHTS.items() for n in names for i in range(3)]


@pytest.mark.parametrize("fn,name,i", PLACES)
def test_sizes_and_strides(fn, name, i):
    """A tensor that is one row short, or whose rows are apart."""
    for f, text in ((lambda t: t[:-1], "are needed"), (lambda t: torch.cat([t, t], 1)[:, :t.shape[1]], "contiguous")):
        a = arguments()
        if i is None:
            a[name] = f(a[name])
        else:
            a[name][i] = f(a[name][i])
        with pytest.raises(ValueError, match=text):
            call(fn, a)


def test_strided_workspace(monkeypatch):
    a = arguments()
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        w4.w4a16_dgrad(a["dY"], M, a["weight"], H, K, G, "asym", a["dX"], torch.zeros(64, 64, dtype=U8)[:, :32])
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 1 if t.dtype == U8 and t.dim() == 1 else 0)
    with pytest.raises(ValueError, match="workspace must be a CUDA tensor"):
        call("dgrad", a)
