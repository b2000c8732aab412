"""CPU-only checks of the gated feed-forward and checkpoint entry points: bad arguments are
refused on the host before anything is launched, the binding refuses tensors that are too small,
and the 64-bit forms that the GPU tests compare with hold against differences."""
import pytest
import torch

import gated_ref as R
from bit_gemm_wise_b200 import w4

FAKE = 0x1000  # 16-byte aligned non-null address; never dereferenced (calls fail validation)
NULL, SHAPE, GROUP, ALIGN, ARG, WORKSPACE = 1, 2, 3, 4, 5, 10


def gated(X=FAKE, M=4, wg=(FAKE, FAKE, FAKE), wu=(FAKE, FAKE, FAKE), H=16, K=128, group=128, mode=1, act=0, Y=FAKE,
          ws=None, n=0):
    return w4.lib().w4a16_gated(X, M, *wg, *wu, H, K, group, mode, act, Y, ws, n, None)


def bwd(dH=FAKE, X=FAKE, X8=None, xs=None, M=4, wg=(FAKE, FAKE, FAKE), wu=(FAKE, FAKE, FAKE), H=16, K=128, group=128,
        mode=1, act=0, dG=FAKE, dU=FAKE, dX=FAKE, ws=None, n=0):
    return w4.lib().w4a16_gated_bwd(dH, X, X8, xs, M, *wg, *wu, H, K, group, mode, act, dG, dU, dX, ws, n, None)


def dgrad(dY=FAKE, M=4, w=(FAKE, FAKE, FAKE), N=16, K=128, group=128, mode=1, dX=FAKE, ws=None, n=0):
    return w4.lib().w4a16_dgrad(dY, M, *w, N, K, group, mode, dX, ws, n, None)


def wgrad(dY=FAKE, X8=FAKE, xs=FAKE, M=4, N=16, K=128, dW=FAKE, flags=0, ws=None, n=0):
    return w4.lib().fp8_ckpt_wgrad(dY, X8, xs, M, N, K, dW, flags, ws, n, None)


WEIGHT_CASES = [
    (dict(K=96, group=64), GROUP), (dict(group=48), GROUP), (dict(K=100, group=32), SHAPE), (dict(K=0), SHAPE),
    (dict(M=0), SHAPE), (dict(M=-1), SHAPE), (dict(M=(1 << 24) + 1), SHAPE), (dict(mode=2), ARG),
]


@pytest.mark.parametrize("fn", [gated, bwd, dgrad])
@pytest.mark.parametrize("kw,code", WEIGHT_CASES)
def test_shapes_groups_and_modes(fn, kw, code):
    assert fn(**kw) == code


def test_products_of_two_dimensions_are_limited():
    """2^40 elements an operand or result: refused before anything is launched."""
    big = 1 << 24
    for fn, kw in [(gated, dict(M=big, H=1 << 17)), (bwd, dict(M=big, H=1 << 17)), (dgrad, dict(M=big, N=1 << 17)),
                   (wgrad, dict(M=big, N=1 << 17)), (gated, dict(M=big, K=1 << 17)), (gated, dict(H=big, K=1 << 17))]:
        assert fn(**kw) == SHAPE
    assert w4.lib().fp8_ckpt_save(FAKE, big, 1 << 17, FAKE, FAKE, None) == SHAPE
    assert w4.lib().fp8_ckpt_load(FAKE, FAKE, big, 1 << 17, FAKE, None) == SHAPE
    assert w4.w4a16_gated_workspace_bytes(big, 1 << 17, 128, 128) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), NULL), (dict(Y=None), NULL), (dict(wg=(None, FAKE, FAKE)), NULL), (dict(wu=(FAKE, None, FAKE)), NULL),
    (dict(wu=(FAKE, FAKE, None)), NULL), (dict(mode=0), ARG), (dict(mode=0, wg=(FAKE, FAKE, None)), ARG),
    (dict(act=2), ARG), (dict(act=-1), ARG), (dict(H=0), SHAPE), (dict(X=FAKE + 2), ALIGN), (dict(Y=FAKE + 8), ALIGN),
    (dict(wg=(FAKE + 4, FAKE, FAKE)), ALIGN), (dict(wu=(FAKE, FAKE, FAKE + 2)), ALIGN), (dict(ws=FAKE + 4, n=1 << 20), ALIGN),
    (dict(M=17), WORKSPACE), (dict(M=17, ws=FAKE, n=64), WORKSPACE),
])
def test_gated_refuses(kw, code):
    assert gated(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dH=None), NULL), (dict(dG=None), NULL), (dict(dU=None), NULL), (dict(X=None), NULL),
    (dict(X=None, X8=FAKE), NULL), (dict(X8=FAKE, xs=FAKE), ARG), (dict(xs=FAKE), ARG), (dict(H=12), SHAPE),
    (dict(act=7), ARG), (dict(dX=FAKE + 4), ALIGN), (dict(dH=FAKE + 2), ALIGN),
    (dict(), WORKSPACE), (dict(X=None, X8=FAKE, xs=FAKE), WORKSPACE), (dict(X=None, X8=FAKE, xs=FAKE, ws=FAKE, n=16), WORKSPACE),
])
def test_gated_bwd_refuses(kw, code):
    assert bwd(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dY=None), NULL), (dict(dX=None), NULL), (dict(w=(FAKE, FAKE, None)), NULL), (dict(mode=0), ARG),
    (dict(N=20), SHAPE), (dict(N=0), SHAPE), (dict(dY=FAKE + 2), ALIGN), (dict(dX=FAKE + 2), ALIGN),
    (dict(), WORKSPACE), (dict(ws=FAKE, n=100), WORKSPACE),
])
def test_dgrad_refuses(kw, code):
    assert dgrad(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dY=None), NULL), (dict(X8=None), NULL), (dict(xs=None), NULL), (dict(dW=None), NULL), (dict(M=0), SHAPE),
    (dict(N=12), SHAPE), (dict(N=0), SHAPE), (dict(K=48), SHAPE), (dict(flags=2), ARG), (dict(dW=FAKE + 4), ALIGN),
])
def test_wgrad_refuses(kw, code):
    assert wgrad(**kw) == code


def test_ckpt_refuses():
    L = w4.lib()
    assert L.fp8_ckpt_save(None, 4, 64, FAKE, FAKE, None) == NULL
    assert L.fp8_ckpt_save(FAKE, 4, 64, FAKE, None, None) == NULL
    assert L.fp8_ckpt_save(FAKE, 0, 64, FAKE, FAKE, None) == SHAPE
    assert L.fp8_ckpt_save(FAKE, 4, 48, FAKE, FAKE, None) == SHAPE
    assert L.fp8_ckpt_save(FAKE, 4, 64, FAKE + 8, FAKE, None) == ALIGN
    assert L.fp8_ckpt_load(FAKE, None, 4, 64, FAKE, None) == NULL
    assert L.fp8_ckpt_load(FAKE, FAKE, 4, 0, FAKE, None) == SHAPE
    assert L.fp8_ckpt_load(FAKE, FAKE + 1, 4, 64, FAKE, None) == ALIGN


def test_workspace_queries_of_refused_shapes_are_zero():
    assert w4.w4a16_gated_workspace_bytes(0, 64, 128, 128) == 0
    assert w4.w4a16_gated_workspace_bytes(64, 64, 96, 64) == 0
    assert w4.w4a16_gated_bwd_workspace_bytes(64, 12, 128, 128, True) == 0
    assert w4.w4a16_dgrad_workspace_bytes(64, 20, 128, 128) == 0
    assert w4.fp8_ckpt_wgrad_workspace_bytes(64, 16, 40) == 0


def test_binding_refuses_host_small_and_strided_tensors():
    M, H, K, g = 4, 16, 128, 128
    wg = R.weight(H, K, g, "asym", 1, "cpu")
    x, y = torch.zeros(M, K, dtype=R.BF16), torch.zeros(M, H, dtype=R.BF16)
    with pytest.raises(ValueError, match="CUDA"):
        w4.w4a16_gated(x, M, wg, wg, H, K, g, "asym", "silu", y)
    with pytest.raises(ValueError, match="CUDA"):
        w4.fp8_ckpt_save(x, M, K, torch.zeros(M, K, dtype=torch.uint8), torch.zeros(M, K // 32, dtype=torch.uint8))


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_reference_gradients_against_differences(name):
    M, H, K, g = 5, 24, 64, 32
    wg, wu = R.weight(H, K, g, "asym", 1, "cpu"), R.weight(H, K, g, "asym", 2, "cpu")
    x, dh = R.rows(M, K, 3, "cpu", std=10.0).double(), R.rows(M, H, 4, "cpu").double()
    _, _, dx = R.gated_grads(x, dh, wg, wu, g, name)
    h = 1e-6
    for i, j in [(0, 0), (2, 17), (4, 63)]:
        p, m = x.clone(), x.clone()
        p[i, j] += h
        m[i, j] -= h
        num = ((R.gated(p, wg, wu, g, name) - R.gated(m, wg, wu, g, name)) * dh).sum() / (2 * h)
        # central differences: O(h^2) truncation and 1e-16 / h rounding, both below 1e-8 here
        assert abs(float(num - dx[i, j])) <= 1e-7 * max(1.0, abs(float(num)))


def test_reference_checkpoint():
    x = torch.tensor([[0.0, 448.0, -449.0, 3.0e38, -1e-38] + [1.0] * 27] * 1, dtype=torch.float32).to(R.BF16)
    s, v = R.save(x)
    back = R.restored(v, s)
    assert int(s[0, 0]) == 127 + 120 and float(back[0, 1]) == 0.0
    y = torch.linspace(-1, 1, 64).reshape(2, 32).to(R.BF16)
    s, v = R.save(y)
    # an E4M3 value is off by at most half a step: 2^-4 relative, or 2^-10 2^e near zero
    err = (R.restored(v, s) - y.double()).abs()
    assert bool((err <= torch.maximum(2.0 ** -4 * y.double().abs(), 2.0 ** -10 * R.two_to(s.long() - 127))).all())
